"""GPU tests of an AdamWGroup's memory beside work that other streams still have to do."""

import pytest

from tests.test_gpu_adamw import HP, _mo, _torch, check, param, snap

pytestmark = pytest.mark.gpu


def busy(torch, count=20):
    """Work that keeps the current stream busy for some milliseconds."""
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(count):
        a @ a


def test_a_groups_table_beside_writes_that_are_still_to_come():
    """Memory freed on the current stream, whose last write waits there, while a group is made and stepped on another
    stream: the table is taken elsewhere, and the step is right."""
    torch, mo = _torch(), _mo()
    p, s = param(5000), torch.cuda.Stream()
    n = mo.AdamWGroup([p], mo.AdamWHyper(**HP)).workspace.numel()
    before = snap(p)
    torch.cuda.synchronize()
    busy(torch)
    late = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    taken = {x.data_ptr() for x in late}
    del late
    group = mo.AdamWGroup([p], mo.AdamWHyper(**HP), stream=s)
    assert group.workspace.data_ptr() not in taken
    group.step(stream=s)
    torch.cuda.synchronize()
    check(p, 0, before, 1)


def test_tensors_of_another_stream_outlive_a_dropped_group():
    """Tensors made on the current stream; a group made, stepped and dropped on another one, whose step still waits."""
    torch, mo = _torch(), _mo()
    p, s = param(5000), torch.cuda.Stream()
    before, want = snap(p), {k: t.clone() for k, t in p.items()}
    places = {t.untyped_storage().data_ptr() for t in p.values()}
    group = mo.AdamWGroup([want], mo.AdamWHyper(**HP))
    group.step()
    check(want, 0, before, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        group = mo.AdamWGroup([p], mo.AdamWHyper(**HP))
        busy(torch)
        group.step()
    sizes = [t.untyped_storage().nbytes() for t in p.values()]
    del group, p
    got = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    if not s.query():
        assert not places & {x.data_ptr() for x in got}
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in got)
