"""The order of a block's calls (MoEBlock): every step's grad_end follows a
grad_begin of its own, also in steps after the first and after a call that
failed. On the CPU with stand-ins for the operators, and on the GPU."""
import types

import pytest
import torch

import pw_inputs
import sparse_shard_exchange_amd as pw


class Memory(str):
    """Stand-in for a tensor, in memory of its own."""

    def untyped_storage(self):
        return types.SimpleNamespace(data_ptr=lambda: self)


class Ops:
    """Stand-in for every operator of a block: results name the call they come from."""
    calls = 0
    fail = None

    def _name(self, what, n):
        if Ops.fail == what:
            raise pw.PwError(pw.PW_ERR_INVALID, what)
        Ops.calls += 1
        return tuple(Memory(f"{what}{Ops.calls}.{i}") for i in range(n))

    def forward(self, *a, **kw):
        return self._name("norm", 2)

    def step(self, *a, **kw):
        return self._name("step", 1)

    def loss(self, *a, **kw):
        return self._name("loss", 3)

    def combine(self, *a, **kw):
        return self._name("combine", 3)

    def dispatch(self, *a, **kw):
        return self._name("dispatch", 2)

    def grad(self, *a, **kw):
        return self._name("grad", 5)


@pytest.fixture
def block():
    b = pw.MoEBlock.__new__(pw.MoEBlock)
    b.moe = Ops()
    b.moe.__dict__.update(logits=0, experts=0, gates=0, src_index=0, offsets=0, w=(0,), static_rows=4,
                          out=Memory("out"), xd=Memory("xd"), y=Memory("y"))
    b.moe.y.shape = (4, 1)
    Ops._buffers = {"h": Memory("h")}
    b.norm_in = b.norm_out = b.balance = b.grads = Ops()
    b.w_in = b.w_out = b.gate = None
    b.h = b._back = b._dgates = None
    Ops.fail = None
    return b


def refused(call, *a):
    with pytest.raises(pw.PwError) as e:
        call(*a)
    return e.value.code


def test_every_step_needs_its_own_grad_begin(block):
    for _ in range(3):
        block.forward(Memory("x"))
        assert refused(block.grad_end, "dxd") == pw.PW_ERR_STATE
        block.grad_begin("dr")
        block.grad_end("dxd")
        block.grad_end("dxd")          # of the same step: the same inputs


@pytest.mark.parametrize("what", ["norm", "step", "loss"])
def test_a_forward_that_failed_leaves_no_step(block, what):
    block.forward(Memory("x"))
    block.grad_begin("dr")
    Ops.fail = what
    assert refused(block.forward, Memory("x")) == pw.PW_ERR_INVALID
    Ops.fail = None
    assert refused(block.grad_begin, "dr") == pw.PW_ERR_STATE
    assert refused(block.grad_end, "dxd") == pw.PW_ERR_STATE


@pytest.mark.parametrize("what", ["grad", "combine"])
def test_a_grad_begin_that_failed_has_no_grad_end(block, what):
    block.forward(Memory("x"))
    block.grad_begin("dr")
    Ops.fail = what
    assert refused(block.grad_begin, "dr") == pw.PW_ERR_INVALID
    Ops.fail = None
    assert refused(block.grad_end, "dxd") == pw.PW_ERR_STATE


@pytest.mark.parametrize("name", ["out", "xd", "y", "h"])
def test_x_in_a_buffer_that_the_step_writes(block, name):
    """The residual and the backward pass read x after the step has written there."""
    block.forward(Memory("x"))
    assert refused(block.forward, Memory(name)) == pw.PW_ERR_INVALID
    block.forward(Memory("x"))


def test_an_x_that_is_updated_in_place_has_no_backward_pass(block):
    block.norm_out.forward = lambda x, **kw: (x if x == "r" else Memory("r"), None)
    block.norm_in = Ops()
    r = block.forward(Memory("x"))[0]
    block.grad_begin("dr")
    block.forward(r)
    assert refused(block.grad_begin, "dr") == pw.PW_ERR_STATE
    assert refused(block.grad_end, "dxd") == pw.PW_ERR_STATE


def test_an_x_that_grad_end_overwrites_is_gone_after_it(block):
    g = Memory("the gradient's buffer")
    block.norm_in = Ops()
    block.norm_in.grad = lambda *a, **kw: (g, None, None, None, None)
    block.forward(Memory("x"))
    block.grad_begin("dr")
    assert block.grad_end("dxd")["x"] is g
    block.forward(g)
    block.grad_begin("dr")
    block.grad_end("dxd")
    assert refused(block.grad_end, "dxd") == pw.PW_ERR_STATE
    assert refused(block.grad_begin, "dr") == pw.PW_ERR_STATE


@pytest.mark.gpu
def test_steps_after_the_first(gpu):
    """A second step's grad_end without a grad_begin is refused, and its
    gradients are those of a fresh block."""
    T, d, E, H = 64, 256, 4, 256
    inp = pw_inputs.moe(T, d, E, H)
    w = inp.w_router.cuda(), inp.w1.cuda(), inp.w2.cuda()
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    one, data = rnd(d), [(rnd(T, d), rnd(T, d), rnd(2 * T, d)) for _ in range(2)]
    new = lambda: gpu.MoEBlock(gpu.MoE(*w, T, num_src_shards=1), one, one, z_coef=0.01)  # noqa: E731

    def backward(block, dr, dxd):
        dy = block.grad_begin(dr)
        return [dy.clone()] + [t.clone() for t in block.grad_end(dxd).values() if t is not None]

    block = new()
    for i, (x, dr, dxd) in enumerate(data):
        f = block.forward(x)[-1]
        with pytest.raises(gpu.PwError) as e:
            block.grad_end(dxd)
        assert e.value.code == gpu.PW_ERR_STATE
        got = backward(block, dr, dxd)
        again = backward(block, dr, dxd)
        fresh = new()
        h = fresh.forward(x)[-1]
        want = backward(fresh, dr, dxd)
        assert len(got) == len(want) == 5
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(got, want, again)), i
        for fut in (f, h):
            gpu.future_wait(fut, 60_000_000_000)


@pytest.mark.gpu
def test_a_block_run_on_its_own_result(gpu):
    """r over x gives the bits of a step on a copy; a backward pass is refused, and so
    is an x that the step overwrites."""
    T, d, E, H = 64, 256, 4, 256
    inp = pw_inputs.moe(T, d, E, H)
    g = torch.Generator().manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    x, one, dr = rnd(T, d), rnd(d), rnd(T, d)
    block = gpu.MoEBlock(gpu.MoE(inp.w_router.cuda(), inp.w1.cuda(), inp.w2.cuda(), T, num_src_shards=1), one, one)
    copy = block.forward(x)[0].clone()
    want = block.forward(copy)[0].clone()
    block.grad_begin(dr)
    r = block.forward(x)[0]
    again, *_, f = block.forward(r)
    assert again.data_ptr() == r.data_ptr() and torch.equal(again, want)
    with pytest.raises(gpu.PwError) as e:
        block.grad_begin(dr)
    assert e.value.code == gpu.PW_ERR_STATE
    for bad in (block.moe.out, block.moe.y[:T], block.moe.xd[:T], block.norm_in._buffers["h"]):
        with pytest.raises(gpu.PwError) as e:
            block.forward(bad)
        assert e.value.code == gpu.PW_ERR_INVALID
    gpu.future_wait(f, 60_000_000_000)
