"""The build says when the compiler gave a kernel another number of registers
than its role split spends (no device work)."""
from bit_kv_cache_centroid_b200 import build

LOG = """ptxas info    : Compiling entry function '_Z16rows_attn_kernelILi64E' for 'sm_100a'
ptxas info    : Function properties for _Z16rows_attn_kernelILi64E
    24 bytes stack frame, 20 bytes spill stores, 32 bytes spill loads
ptxas info    : Used {} registers, used 3 barriers, 24 bytes cumulative stack size
ptxas info    : Compiling entry function '_Z14rows_merge_cutILi64E' for 'sm_100a'
ptxas info    : Function properties for _Z14rows_merge_cutILi64E
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 40 registers, used 0 barriers
"""


def test_other_counts_are_found():
    assert build.wrong_registers("rows_attn.cu", LOG.format(72)) == []
    assert build.wrong_registers("rows_attn.cu", LOG.format(71)) == [("_Z16rows_attn_kernelILi64E", 71)]
