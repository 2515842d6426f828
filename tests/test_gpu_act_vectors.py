"""GPU tests of block norms whose vectors move between calls."""
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
