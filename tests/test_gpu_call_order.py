"""Calls that write what the next call reads, with no other kernel between them: every
call has to see what the one before it wrote, bit for bit what it sees when the host
waits between them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

Hq, Hkv, d = 32, 8, 128


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from long_context_sparse_score_gb300 import _build
    _build.build()
    from long_context_sparse_score_gb300 import hashattn
    hashattn.lib()
    return hashattn


class Loop:
    """A serving loop over one cache [B, Hkv, cap, d]: each step appends `new` tokens to every
    sequence and attends with the last of them. All inputs are made beforehand."""

    def __init__(self, H, B, cap, start, steps, new=1):
        self.H, self.B, self.cap, self.new = H, B, cap, new
        g = torch.Generator(device="cuda").manual_seed(B + cap)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.K0, self.V0 = rand(B, Hkv, cap, d), rand(B, Hkv, cap, d)
        self.W = torch.randn(Hkv, 32, d, generator=g, device="cuda")
        self.table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
        self.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * new
        self.rope = H.rope(torch.tensor([10000.0 ** (-2.0 * i / d) for i in range(d // 2)], device="cuda"))
        self.rows = [tuple(rand(B * new, h, d) for h in (Hq, Hkv, Hkv)) for _ in range(steps)]
        self.lens = [torch.full((B,), start + (i + 1) * new, dtype=torch.int32, device="cuda") for i in range(steps)]
        self.pos = [x - 1 for x in self.lens]
        K, V, sig, shape = self.fresh()
        for at in range(start):
            H.hash_attn_encode_keys(shape, K, self.W, torch.full((B,), at, dtype=torch.int32, device="cuda"), sig)
        self.sig0 = sig
        self.m = 64
        sizes = [H.hash_attn_workspace_size(shape, m, 4, 8) for m in (self.m, cap)]
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
        H.hash_attn_workspace_init(self.ws)
        self.ws2 = torch.empty_like(self.ws)
        H.hash_attn_workspace_init(self.ws2)
        tok = H.make_tokens(*self.rows[0], B, out_dtype=torch.bfloat16)
        self.wp = torch.zeros(H.hash_attn_packed_workspace_size(tok), dtype=torch.uint8, device="cuda")

    def fresh(self):
        sig = self.sig0.clone() if hasattr(self, "sig0") else torch.zeros(self.B, Hkv, self.cap, dtype=torch.int32, device="cuda")
        K, V = self.K0.clone(), self.V0.clone()
        return K, V, sig, self.H.make_shape(self.rows[0][0][:self.B], K, V, sig)

    def run(self, chain, wait, q_sigs=None):
        """The outputs of every step; `wait` between two calls."""
        H, B = self.H, self.B
        K, V, sig, shape = self.fresh()
        cache = H.make_cache(K, V, self.table, sig)
        n = len(self.rows)
        toks = [H.make_tokens(*r, B, out_dtype=torch.bfloat16) for r in self.rows]
        # one set of buffers for all steps: a step that reads too early finds the last step's values
        qo = torch.zeros(B * self.new, Hq, d, dtype=torch.bfloat16, device="cuda")
        q = qo[self.new - 1::self.new]
        q_sig = torch.zeros(B, Hq, dtype=torch.int32, device="cuda")
        outs = [(torch.full((B, Hq, d), float("nan"), device="cuda"), torch.full((B, Hq), float("nan"), device="cuda")) for _ in range(n)]
        couts = [(torch.empty_like(qo), torch.empty(qo.shape[:2], device="cuda")) for _ in range(n)]
        douts = [tuple(torch.full_like(x, float("nan")) for x in o) for o in outs]
        sigs = []
        st = torch.cuda.current_stream()
        shape = H.make_shape(q, K, V, sig)
        st.synchronize()
        if not wait:
            torch.cuda._sleep(2_000_000)  # the calls queue up behind it
        for i, (r, tok, lens) in enumerate(zip(self.rows, toks, self.lens)):
            codes = dict(W=self.W, k_sig=sig) if "codes" in chain else {}
            H.hash_attn_append(tok, cache, *r, self.table, self.cu, lens, qo, K, V, rope=self.rope, stream=st, **codes)
            if "keys" in chain:
                wait and st.synchronize()
                H.hash_attn_encode_keys(shape, K, self.W, self.pos[i], sig, stream=st)
            if "queries" in chain:
                wait and st.synchronize()
                H.hash_attn_encode_queries(shape, q, self.W, q_sig, stream=st)
                sigs.append(q_sig.clone())
            if "chunk" in chain:
                wait and st.synchronize()
                H.hash_attn_chunk(tok, cache, qo, K, V, self.table, self.cu, lens, *couts[i], workspace=self.wp, stream=st)
            wait and st.synchronize()
            if "both" in chain:  # two decode calls in turn, each with a workspace of its own
                H.hash_attn_decode(shape, q, None, None, K, V, lens, None, self.cap, 4, 8, *douts[i], workspace=self.ws2, stream=st)
                wait and st.synchronize()
            if "dense" in chain:
                H.hash_attn_decode(shape, q, None, None, K, V, lens, None, self.cap, 4, 8, *outs[i], workspace=self.ws, stream=st)
            else:
                H.hash_attn_decode(shape, q, q_sig if q_sigs is None else q_sigs[i], sig, K, V, lens, None, self.m, 4, 8, *outs[i],
                                   workspace=self.ws, stream=st)
            wait and st.synchronize()
        assert all(H.hash_attn_device_status(w)[0] == 0 for w in (self.ws, self.ws2, self.wp))
        more = (couts if "chunk" in chain else []) + (douts if "both" in chain else [])
        return [t for o in outs + more for t in o] + [K, V, sig], sigs


CHAINS = {
    "append-dense": ("dense",),
    "append-chunk-dense": ("chunk", "dense"),
    "append-codes-dense": ("codes", "dense"),
    "append-codes-sparse": ("codes",),
    "append-chunk-sparse": ("codes", "chunk"),
    "append-keys-sparse": ("keys",),
    "append-dense-sparse": ("codes", "both"),
    "append-chunk-dense-sparse": ("codes", "chunk", "both"),
    "append-dense-dense": ("both", "dense"),
}


# the last with a grid of decode CTAs that leaves room for the others beside it, and more tokens a step
@pytest.mark.parametrize("B,cap,start,new", [(8, 256, 100, 1), (64, 128, 40, 1), (2, 8200, 20, 7)])
@pytest.mark.parametrize("chain", CHAINS.values(), ids=CHAINS)
def test_a_call_sees_what_the_call_before_it_wrote(H, chain, B, cap, start, new):
    loop = Loop(H, B, cap, start, 6, new)
    # the queries' codes of every step are there beforehand, so that nothing runs between append and decode
    q_sigs = None if "dense" in chain else loop.run(chain + ("queries",), True)[1]
    want, _ = loop.run(chain, True, q_sigs)
    got, _ = loop.run(chain, False, q_sigs)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), f"{chain}: result {i} of {len(want)}"
    assert all(torch.isfinite(x).all() for x in want[:12])
