"""A workspace query answers for its own M: fewer rows may need more, as the header says, and the binding asks again."""

import os
import re

from qlora_fine_tuning_nf4_b200 import build, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_fewer_rows_may_need_more():
    build.build()
    assert ops.fp8_matmul_workspace_bytes(8192, 4096, 4096) == 256
    assert ops.fp8_matmul_workspace_bytes(128, 4096, 4096) == 256 + 8 * 2 ** 20
    assert ops.qlora_linear8_workspace_bytes(300, 4096, 4096) < ops.qlora_linear8_workspace_bytes(256, 4096, 4096)


def test_the_header_says_so():
    text = open(os.path.join(ROOT, "include", "qlora.h")).read()
    text = re.sub(r"\s*\n \*\s*", " ", text)
    assert "A query answers for the M it is asked about. A smaller M may need more" in re.sub(r" +", " ", text)
