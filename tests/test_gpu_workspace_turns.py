"""One workspace serves every entry point and path on its shape in turn: what must be zero between
calls lies at the same place for the decode on virtual KV heads (more than four query heads per KV
head, or a small grid) and for the calls on the real ones."""
import pytest
import torch

import gpu_helpers as GH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    hashattn.lib()


CASES = [
    # name, B, Hq, Hkv, n_cap, lens, m
    ("small-grid-g4", 1, 8, 2, 9000, [9000], 300),
    ("g8", 2, 16, 2, 9000, [9000, 4000], 500),
    ("g16", 3, 16, 1, 20000, [20000, 1, 15000], 700),
    ("g5", 2, 10, 2, 3000, [3000, 2999], 100),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_entry_points_take_turns_on_a_workspace(case):
    from long_context_sparse_score_gb300 import workloads as W
    H = GH.ha()
    _, B, Hq, Hkv, n_cap, lens, m = case
    w = W.make_gqa(21, B=B, Hq=Hq, Hkv=Hkv, d=128, n_cap=n_cap, seq_lens=lens, m=m, n_sink=16, n_local=64, device="cuda")
    shape = H.make_shape(w.q, w.K, w.V, w.k_sig, batch=B)
    gen = torch.Generator(device="cuda").manual_seed(5)
    words = 4
    wide_k = torch.randint(-2**31, 2**31 - 1, (B, Hkv, n_cap, words), generator=gen, device="cuda").int()
    wide_q = torch.randint(-2**31, 2**31 - 1, (B, Hq, words), generator=gen, device="cuda").int()
    wide_shape = H.make_shape(w.q, w.K, w.V, wide_k, batch=B)
    opts = H.select_opts(None, False, words)
    size = max(H.hash_attn_workspace_size(shape, n_cap, 16, 64), H.hash_attn_workspace_size(shape, m, 16, 64),
               H.hash_attn_workspace_size_ex(wide_shape, m, 16, 64, opts))
    cap = H.hash_attn_select_capacity(n_cap, m, 16, 64)

    def new_ws():
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        H.hash_attn_workspace_init(ws)
        return ws

    def results(*shapes):
        return [torch.full(s, float("nan"), device="cuda") for s in shapes]

    def decode(ws):
        out, lse = results((B, Hq, 128), (B, Hq))
        H.hash_attn_decode(shape, w.q, w.q_sig, w.k_sig, w.K, w.V, w.seq_lens, None, m, 16, 64, out, lse, workspace=ws)
        return out, lse

    def with_lists(ws):
        out, lse = results((B, Hq, 128), (B, Hq))
        idx, cnt = torch.empty(B, Hq, cap, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, dtype=torch.int32, device="cuda")
        H.hash_attn_decode(shape, w.q, w.q_sig, w.k_sig, w.K, w.V, w.seq_lens, None, m, 16, 64, out, lse, idx, cnt, workspace=ws)
        return out, lse, idx, cnt

    def dense(ws):
        out, lse = results((B, Hq, 128), (B, Hq))
        H.hash_attn_decode(shape, w.q, None, None, w.K, w.V, w.seq_lens, None, n_cap, 16, 64, out, lse, workspace=ws)
        return out, lse

    def select_and_gather(ws):
        out, lse = results((B, Hq, 128), (B, Hq))
        idx, cnt = torch.empty(B, Hq, cap, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, dtype=torch.int32, device="cuda")
        H.hash_attn_select(shape, w.q_sig, w.k_sig, w.seq_lens, None, m, 16, 64, idx, cnt, workspace=ws)
        H.hash_attn_gather_att(shape, w.q, w.K, w.V, w.seq_lens, idx, cap, cnt, out, lse, workspace=ws)
        return out, lse, idx, cnt

    def wide(ws):
        out, lse = results((B, Hq, 128), (B, Hq))
        H.hash_attn_decode_ex(wide_shape, w.q, wide_q, wide_k, w.K, w.V, w.seq_lens, None, m, 16, 64, opts, out, lse, workspace=ws)
        return out, lse

    calls = [decode, with_lists, dense, select_and_gather, wide]
    want = {c: c(new_ws()) for c in calls}
    ws = new_ws()
    for first in calls:
        for second in calls:
            for c in (first, second):
                got = c(ws)
                assert H.hash_attn_device_status(ws) == (0, 0), f"{c.__name__} ({first.__name__}, {second.__name__})"
                for a, b in zip(got, want[c]):
                    assert torch.equal(a, b), f"{c.__name__} ({first.__name__}, {second.__name__})"
