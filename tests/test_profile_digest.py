"""The sources that the profiles' digests are over: a file of the block operators
left out of their list would count as a matmul kernel, and make the matmul's
counters look out of date."""
import os
import re

from vq_dequant_matmul_gemv_amd import profsum


def test_block_sources_are_all_listed():
    names = os.listdir(os.path.join(profsum.HERE, "csrc"))
    assert {n for n in names if re.match(r"vq_(block|fp8|mx4|norm|router|store)", n)} == set(profsum.BLOCK_SOURCES)
