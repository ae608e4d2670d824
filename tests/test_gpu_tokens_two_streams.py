"""Two contexts on streams of their own, whose calls run at the same time on the same SMs: each gives what it gives alone."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [1, 24, 300, 600])
def test_two_contexts_at_once(S):
    streams = [torch.cuda.Stream() for _ in range(2)]
    sides, handles = [B.coli_init(0, s) for s in streams], []
    g = torch.Generator(device="cuda").manual_seed(S)
    freqs = B.coli_rotary_freqs(64)
    V, I = 6001, 1280
    try:
        work = []
        for c in sides:
            h = B.coli_dense_upload(c, (0.05 * torch.randn(V, I, device="cuda", generator=g)).bfloat16())
            handles.append(h)
            work.append((c, h, torch.randn(S, 20, 64, device="cuda", generator=g),
                         torch.arange(S, dtype=torch.int32, device="cuda"), torch.randint(0, V, (S, 1), dtype=torch.int32, device="cuda", generator=g)))

        def chain(c, h, x, positions, tokens):
            turned, logits = torch.empty_like(x), torch.empty(S, V, device="cuda")
            out = dict(logp=torch.empty(S, 1, device="cuda"), entropy=torch.empty(S, device="cuda"),
                       top_id=torch.empty(S, 8, dtype=torch.int32, device="cuda"), top_logp=torch.empty(S, 8, device="cuda"))
            B.coli_rotary(c, x, None, freqs, turned, None, positions=positions)
            B.coli_dense_linear(c, h, turned.view(S, I), logits, act="silu")
            B.coli_logprobs(c, logits, tokens=tokens, **out)
            return [turned, logits, *out.values()]

        torch.cuda.synchronize()
        alone = []
        for s, w in zip(streams, work):
            with torch.cuda.stream(s):
                alone.append(chain(*w))
            torch.cuda.synchronize()
        results = [[], []]
        for _ in range(40):
            for i, (s, w) in enumerate(zip(streams, work)):
                with torch.cuda.stream(s):
                    results[i].append(chain(*w))
        torch.cuda.synchronize()
        for one, many in zip(alone, results):
            for r in many:
                assert all(torch.equal(a, b) for a, b in zip(one, r))
        assert [B.coli_check_error(c) for c in sides] == [0, 0]
    finally:
        for c, h in zip(sides, handles):
            B.coli_dense_free(c, h)
        for c in sides:
            B.coli_destroy(c)
