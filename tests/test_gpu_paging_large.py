"""Batch plan and cache write at sizes where a thread takes more than one entry,
row or group of words."""
import pytest

from tests.test_gpu_paging import draw_plan, mla, plan_reference, run_plan, same  # noqa: F401

pytestmark = pytest.mark.gpu


def test_plan_of_more_rows_and_shared_entries_than_threads(mla):  # noqa: F811
    import torch
    threads = 512 * torch.cuda.get_device_properties(0).multi_processor_count
    c = draw_plan(71, B=1024, bs=16, ctx_hi=100, new_hi=200, nshared=90, pad=5003)
    assert c["T"] > threads and 1024 * 90 > threads
    ref = plan_reference(**c)
    got, err = run_plan(mla, **c)
    assert err == mla.MLA_OK and not ref["error"]
    same(got, ref)


def test_plan_of_more_taken_pages_than_threads(mla):  # noqa: F811
    import torch
    threads = 512 * torch.cuda.get_device_properties(0).multi_processor_count
    c = draw_plan(72, B=300, bs=1, ctx_hi=30, new_hi=600, nshared=2, pad=77)
    ref = plan_reference(**c)
    assert int(ref["used"][0]) > threads and not ref["error"]
    got, err = run_plan(mla, **c)
    assert err == mla.MLA_OK
    same(got, ref)


@pytest.mark.parametrize("d_c,d_r,dtype,T", [(512, 64, "bf16", 20011), (512, 64, "fp32", 9001), (13, 6, "bf16", 70001)])
def test_cache_write_of_more_words_than_one_pass(mla, d_c, d_r, dtype, T):  # noqa: F811
    import torch
    p = mla.dims(256, 4, 32, d_c, 96, d_r, dtype=dtype)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    it = torch.int16 if dtype == "bf16" else torch.int32
    D = d_c + d_r
    row = D * dt.itemsize
    vec = row // (16 if row % 16 == 0 else 4 if row % 4 == 0 else 2)
    assert T * vec > 8 * torch.cuda.get_device_properties(0).multi_processor_count * 256 * 4  # one pass
    g = torch.Generator().manual_seed(T)
    nb = T // 64 + 3
    rows, data = torch.randn((T, D), generator=g).to(dt), torch.randn((nb, 64, D), generator=g).to(dt)
    slots = torch.randperm(nb * 64, generator=g)[:T].clone()
    slots[torch.randperm(T, generator=g)[:97]] = -1
    slots[-1] = -1
    want, keep = data.clone().view(-1, D), slots >= 0
    want[slots[keep]] = rows[keep]
    dev = data.cuda()
    mla.mla_cache_write(p, rows.cuda(), slots.cuda(), mla.Cache(dev, torch.zeros((1, nb), dtype=torch.int32, device="cuda")))
    assert mla.mla_get_device_error() == mla.MLA_OK
    assert torch.equal(dev.cpu().view(it), want.view(dev.shape).view(it))
