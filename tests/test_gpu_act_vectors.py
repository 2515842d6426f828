"""GPU tests of the memory that the activation checkpoints' calls use: vectors that
move between calls, workspaces of a call's own."""
import pytest
import torch

from act_util import codes, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ps():
    import precision_state_amd as ps
    return ps


@pytest.mark.parametrize("how", ["data", "storage"])
def test_vectors_are_read_where_they_are(ps, how):
    """Other memory by `.data`, or a storage that is released and comes back elsewhere, as sharded training does: the
    results are those of a norm that was made of the new values."""
    rows, cols = 40, 264
    g = gen(3)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, y, dn = r(rows, cols), r(rows, cols), r(rows, cols)
    names = ("post_weight", "gate", "mul", "add")

    def run(norm):
        n, h, dx, dy = (torch.empty_like(x) for _ in range(4))
        s = dict(h_code=codes(rows, cols), h_rstd=torch.empty(rows, device="cuda"), y_code=codes(rows, cols),
                 y_rstd=torch.empty(rows, device="cuda"))
        ps.block_norm_forward(norm, x, n, y=y, h=h, **s)
        grads = {f"d_{k}": torch.empty(cols, device="cuda") for k in names}
        ps.block_norm_backward(norm, dn, dx=dx, dy=dy, **s, **grads)
        return [n, h, dx, dy, *grads.values()]
    v = {k: r(cols) for k in names}
    norm = ps.BlockNorm(post_norm=ps.NORM_RMS, **v)
    run(norm)
    new = {k: r(cols) for k in names}
    for k in names:
        if how == "data":
            v[k].data = new[k].clone()
        else:
            storage, size = v[k].untyped_storage(), v[k].untyped_storage().nbytes()
            torch.cuda.synchronize()
            storage.resize_(0)
            hold = torch.full((cols,), float("nan"), device="cuda")     # takes the place that was given up
            storage.resize_(size)
            v[k].copy_(new[k])
            new[k + "_hold"] = hold
    want = run(ps.BlockNorm(post_norm=ps.NORM_RMS, **{k: new[k] for k in names}))
    got = run(norm)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_workspace_belongs_to_the_stream_of_its_call(ps, monkeypatch):
    """Given back, it may be handed out again in that stream's order only; the default stream's number is 0."""
    device = torch.device("cuda", 0)
    side = torch.cuda.Stream()
    seen = []
    empty = torch.empty

    def record(*a, **kw):
        seen.append(torch.cuda.current_stream(device).cuda_stream)
        return empty(*a, **kw)
    dy, code = torch.ones(2000, 96, dtype=torch.bfloat16, device=device), torch.full((2000, 640), 0x38, dtype=torch.uint8, device=device)
    w = torch.empty(96, 640, device=device)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", record)
    default = torch.cuda.default_stream(device).cuda_stream
    for stream, want in ((0, default), (None, default), (torch.cuda.default_stream(device), default),
                         (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
        w.zero_()
        torch.cuda.synchronize()
        seen.clear()
        ps.linear_wgrad(dy, code, w, stream=stream)
        torch.cuda.synchronize()
        assert seen == [want], stream
        assert (w == 2000).all()
    with torch.cuda.stream(side):                       # 0 is the default stream, not the current one
        seen.clear()
        ps.linear_wgrad(dy, code, w, stream=0)
        assert seen == [default]
    torch.cuda.synchronize()
