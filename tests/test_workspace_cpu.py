"""Workspace sizes on the host: one workspace serves every call of up to the tokens it was sized for."""
import ctypes

import pytest

import mixture_experts_histogram_b200 as m
from conftest import cuda_available
from mixture_experts_histogram_b200 import build

# H, E, k, S, I
LAYERS = [(4096, 352, 8, 1, 1536), (1024, 16, 2, 1, 512), (512, 5, 1, 0, 1024), (16384, 64, 4, 1, 512)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return m.load()


@pytest.mark.parametrize("w", range(4))
@pytest.mark.parametrize("layer", LAYERS)
def test_size_never_falls(lib, w, layer):
    cfg = m.make_config(*layer[:4], layer[4], w)
    sizes = [m.moe_workspace_bytes(cfg, T) for T in range(65)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def calls(lib, cfg, T, nb):
    """Every entry point with a workspace of nb bytes, all else in order (its buffers do not exist)."""
    w = m.moe_weights(*[1 << 20 for _ in m.WEIGHT_FIELDS])
    c, w = ctypes.byref(cfg), ctypes.byref(w)
    R = (cfg.top_k + cfg.n_shared) * T
    yield "moe_forward", lib.moe_forward(c, T, 1024, w, 2048, None, None, 4096, nb, None)
    yield "moe_forward_host", lib.moe_forward_host(c, T, 1024, w, 2048, 4096, nb, None)
    yield "moe_forward_host_async", lib.moe_forward_host_async(c, T, 1024, w, 2048, 4096, nb, None)
    yield "moe_route", lib.moe_route(c, T, 1024, 2048, None, 4096, 8192, None, 4096, nb, None)
    yield "moe_permute", lib.moe_permute(c, T, 1024, 2048, 4096, 8192, 16384, 4096, nb, None)
    yield "moe_experts", lib.moe_experts(c, T, 1024, 2048, 4096, w, 8192, 16384, 4096, nb, None)
    yield "moe_forward_ep_partial", lib.moe_forward_ep_partial(c, T, 1024, w, 0, cfg.n_experts, 0, T, 2048, None, None,
                                                               4096, nb, None)
    yield "moe_grouped_gemm", lib.moe_grouped_gemm(c, m.MOE_STAGE_DOWN, R, 1024, 2048, 4096, w, None, 8192, None, 4096,
                                                   nb, None)
    if T <= m.MOE_FEW_MAX_TOKENS:
        yield "moe_forward_few", lib.moe_forward_few(c, T, 1024, w, 2048, None, None, 4096, nb, None)


@pytest.mark.skipif(cuda_available(), reason="calls with buffers that do not exist end at the missing device")
@pytest.mark.parametrize("w", range(4))
def test_one_workspace_for_fewer_tokens(lib, w):
    """A workspace for 16 tokens is large enough for 1 to 16 (no call gets far: there is no device)."""
    cfg = m.make_config(4096, 352, 8, 1, 1536, w)
    nb = m.moe_workspace_bytes(cfg, 16)
    for T in range(1, 17):
        for name, rc in calls(lib, cfg, T, nb):
            assert rc == m.MOE_ERR_CUDA, (name, T, rc)


@pytest.mark.skipif(cuda_available(), reason="calls with buffers that do not exist end at the missing device")
@pytest.mark.parametrize("w,before", [(0, 1_746_944), (1, 1_406_976), (2, 1_746_944)])
def test_few_token_scratch_is_asked_for_by_its_call_only(lib, w, before):
    """8 tokens of the 352-expert layer: what the other entry points use is a third of what h of the
    few-token layer takes."""
    cfg = m.make_config(4096, 352, 8, 1, 1536, w)
    for name, rc in calls(lib, cfg, 8, before):
        assert rc == (m.MOE_ERR_WORKSPACE_TOO_SMALL if name == "moe_forward_few" else m.MOE_ERR_CUDA), (name, rc)


@pytest.mark.parametrize("w", range(4))
@pytest.mark.parametrize("layer", LAYERS + [(4096, 1, 1, 0, 11264), (128, 1, 1, 0, 128), (2048, 512, 16, 1, 512)])
def test_size_never_falls_where_splits_end(lib, w, layer):
    """Counts around those at which the router's logits or the down GEMM's sums are split less, and a few
    far ones."""
    if w >= 2 and (layer[0] % 512 or layer[4] % 512):
        pytest.skip("not a shape of this storage")
    cfg = m.make_config(*layer[:4], layer[4], w)
    tokens = sorted({t for n in range(1, 160) for t in (128 * n, 128 * n + 1)} | set(range(1, 300)) | {1 << 18, 1 << 20})
    sizes = [m.moe_workspace_bytes(cfg, T) for T in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.skipif(cuda_available(), reason="calls with buffers that do not exist end at the missing device")
def test_one_workspace_where_splits_end(lib):
    """1152 tokens take more partial logits than 1153; the larger batch's workspace serves them."""
    cfg = m.make_config(512, 512, 1, 0, 512, 3)
    nb = m.moe_workspace_bytes(cfg, 1153)
    for T in (1, 8, 9, 1151, 1152, 1153):
        for name, rc in calls(lib, cfg, T, nb):
            assert rc == m.MOE_ERR_CUDA, (name, T, rc)
