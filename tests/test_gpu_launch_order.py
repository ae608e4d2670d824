"""Expert calls straight after the calls that write their input: kernels overlap at their ends (programmatic dependent
launch), and what an expert call reads has to be what the call before it wrote."""
import pytest
import torch

from int4_grouped_expert_router_gb300 import binding as B
from int4_grouped_expert_router_gb300.workload import DeviceLayer, LayerConfig
from gpu_util import Ctx
from kv4_util import Batch

pytestmark = pytest.mark.gpu

ROUNDS = 40
# name: (environment, D, tokens): the streaming kernel, the gate/up and down kernels, the one-kernel form, a few tokens
EXPERTS = {"stream": ({}, 1024, 1), "two kernels": (dict(COLI_DECODE_STREAM=0), 1024, 1),
           "one kernel": (dict(COLI_DECODE_FUSED=1), 1024, 1), "small": ({}, 256, 1), "three tokens": ({}, 1024, 3)}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Setup:
    def __init__(self, name, dtype="f32"):
        env, self.D, self.S = EXPERTS[name]
        self.ctx = Ctx.with_env(**env).ctx
        self.cfg = LayerConfig("order", D=self.D, I=128, E=8, K=2, S=self.S, x_dtype=dtype)
        self.layer = DeviceLayer(self.ctx, self.cfg)
        self.routes = self.layer.outputs()
        x = torch.randn(self.S, self.D, device="cuda", generator=gen(1))
        B.coli_router_select(self.ctx, x, self.layer.Wr, self.layer.bias, self.cfg.K, 0.0, True, 1.0, self.routes["idx"],
                             self.routes["w"], self.routes["n_sel"])
        assert B.coli_check_error(self.ctx) == 0

    def experts(self, x, y):
        B.coli_expert_group(self.ctx, x, self.routes["idx"], self.routes["w"], self.routes["n_sel"], self.cfg.K, None, y)

    def compare(self, x, write):
        """write(i) fills x with round i's input by a library call; the experts' results with and without waiting."""
        results = []
        for wait in (True, False):
            ys = [torch.empty(self.S, self.D, dtype=x.dtype, device="cuda") for _ in range(ROUNDS)]
            torch.cuda.synchronize()
            for i in range(ROUNDS):
                write(i)
                if wait:
                    torch.cuda.synchronize()
                self.experts(x, ys[i])
            assert B.coli_check_error(self.ctx) == 0
            results.append(torch.stack(ys))
        assert torch.equal(*results)
        assert not torch.equal(results[0][0], results[0][1])

    def close(self):
        self.layer.free()
        B.coli_destroy(self.ctx)


@pytest.mark.parametrize("rows", ["few", "many"])
@pytest.mark.parametrize("name", list(EXPERTS))
def test_a_norms_output(name, rows):
    s = Setup(name)
    try:
        R = s.S if rows == "few" else 4096  # of many rows the experts take the last, which the norm writes last
        blocks = torch.randn(8, R, s.D, device="cuda", generator=gen(2))
        w = torch.ones(s.D, device="cuda")
        h, x = torch.empty(R, s.D, device="cuda"), torch.zeros(R, s.D, device="cuda")
        s.compare(x[R - s.S:], lambda i: B.coli_norm_residual(s.ctx, blocks[i % 8], None, None, 1.0 + i, None, w, 1e-5, h, x))
    finally:
        s.close()


@pytest.mark.parametrize("name", ["stream", "two kernels", "three tokens"])
@pytest.mark.parametrize("form", ["attention", "prompt attention", "read"])
def test_an_attentions_output_and_rows_read_back(name, form):
    s = Setup(name, "bf16")
    try:
        m = 1 if form == "attention" else 64
        b = Batch(s.ctx, [3000, 500, 700], 8 if form == "read" else 2, 128, 64, 64, "bf16")
        qs = [b.queries([m] * 3, 8, seed=k)[1] for k in range(8)]
        out = torch.zeros_like(qs[0])
        start = None if m == 1 else torch.from_numpy(b.q_start).cuda()
        lens = [torch.tensor([500 + 300 * k, 500, 700 - k], dtype=torch.int32, device="cuda") for k in range(8)]
        v = torch.empty_like(out)

        def write(i):
            if form == "read":
                B.coli_kv4_read(s.ctx, b.cache, v, out, lens[i % 8], b.table, start)
            else:
                B.coli_kv4_attention(s.ctx, b.cache, qs[i % 8], lens[i % 8], b.table, out, q_start=start)

        s.compare(out.view(-1, s.D)[-s.S:], write)
    finally:
        s.close()


def test_an_input_overwritten_between_the_router_and_the_experts():
    """Router on x, then a norm into the same x, then the experts; and issues of one round on the router's x."""
    s = Setup("stream")
    try:
        blocks = torch.randn(8, 1, s.D, device="cuda", generator=gen(3))
        w = torch.ones(s.D, device="cuda")
        x = torch.ones(1, s.D, device="cuda")
        out = s.layer.outputs()

        def write(i):
            B.coli_router_select(s.ctx, x, s.layer.Wr, s.layer.bias, 2, 0.0, True, 1.0, out["idx"], out["w"], out["n_sel"])
            B.coli_norm_residual(s.ctx, blocks[i % 8], None, None, 1.0 + i, None, w, 1e-5, None, x)

        s.compare(x, write)
        r, y, z = s.routes, torch.empty(1, s.D, device="cuda"), torch.empty(1, s.D, device="cuda")
        for i in range(ROUNDS):
            write(i)
            s.layer.step(x, None, out)
            B.coli_router_select(s.ctx, x, s.layer.Wr, s.layer.bias, 2, 0.0, True, 2.5, r["idx"], r["w"], r["n_sel"])
            for k in range(2):
                B.coli_expert_group_issue(s.ctx, x, r["idx"][:, k:k + 1].contiguous(), r["w"][:, k:k + 1].contiguous(), None, 1)
            B.coli_expert_group_take(s.ctx, None, z)
            torch.cuda.synchronize()
            assert torch.allclose(out["y"], z, rtol=1e-5, atol=1e-5)
        assert B.coli_check_error(s.ctx) == 0
    finally:
        s.close()
