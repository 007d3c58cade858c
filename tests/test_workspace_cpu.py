"""The head that every workspace starts with (no GPU needed)."""
import os
import re

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def q():
    from quantized_linear_layers_token_b200 import build, qlin
    build.build()
    return qlin


def test_head_is_the_headers(q):
    with open(os.path.join(ROOT, "include", "qlin.h")) as f:
        assert int(re.search(r"#define QLIN_WORKSPACE_HEAD (\d+)", f.read()).group(1)) == q.QLIN_WORKSPACE_HEAD


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("M", [0, 1, 40, 300, 5000])
def test_sizes_hold_the_head(q, fmt, M):
    for nO in (0, 5, 300):
        w = q.qlin_weights_bind(512, 1040, fmt, nO, 1 << 20, q.qlin_weights_bytes(512, 1040, fmt, nO))
        sizes = [q.qlin_quant_act_workspace(M, w), q.qlin_gemm_workspace(M, w), q.qlin_backward_dx_workspace(M, w),
                 q.qlin_backward_act_workspace(M, w), q.qlin_backward_gated_workspace(M, w),
                 q.qlin_norm_backward_workspace(M, 512)]
        always = [q.qlin_forward_workspace(M, w), q.qlin_forward_act_workspace(M, w), q.qlin_forward_gated_workspace(M, w)]
        if M <= 64:
            always.append(q.qlin_forward_grouped_workspace([w], M))
        assert all(n == 0 or n >= q.QLIN_WORKSPACE_HEAD for n in sizes)
        assert all(n >= q.QLIN_WORKSPACE_HEAD for n in always)
        assert (sizes[0] > 0) == (nO > 0)
