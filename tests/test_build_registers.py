"""The build's check of the registers that the prefix kernel's exchange counts on (CPU)."""
import os

import pytest

import __graft_entry__

SOURCE = os.path.join(__graft_entry__.ROOT, "paged_kv_cache_476_b200", "csrc", "shared.cu")
LOG = """ptxas info    : Compiling entry function '_ZN3pkv2sh19shared_merge_kernelILi64ELi8EEEv' for 'sm_100a'
ptxas info    : Used 40 registers, used 1 barriers, 9216 bytes smem
ptxas info    : Compiling entry function '_ZN3pkv2sh13prefix_kernelILi128ELi0EEEv' for 'sm_100a'
ptxas info    : Used 80 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN3pkv2sh13prefix_kernelILi128ELi1EEEv' for 'sm_100a'
ptxas info    : Used {} registers, used 1 barriers
"""


@pytest.fixture(scope="module")
def check():
    with open(SOURCE) as f:
        source = f.read()
    builder = __graft_entry__._builder()
    return lambda log, source=source: builder.check_registers(source, log)


def test_enough(check):
    check(LOG.format(96))
    check(LOG.format(104))
    check("", "constexpr int kOther = 3;")


@pytest.mark.parametrize("n", [88, 64, 9])
def test_too_few(check, n):
    with pytest.raises(RuntimeError, match=f"{n} registers"):
        check(LOG.format(n))


def test_nothing_to_look_at(check):
    with pytest.raises(RuntimeError):
        check("")
