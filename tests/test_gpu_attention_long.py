"""The attention kernel against 64 bits with a bound that is far below the
outputs (attention_cases.py; test_attention_bounds.py shows what it rejects), in
every form: after many steps of its loop, with items of hundreds of pages (a
wave holds 64 page ids and takes the next ones as it goes) and of 9 to 39 chunks
a wave, and over short rows."""

import numpy as np
import pytest
import torch

import int4_group_quantized_q4_amd as w4
import oracle
from attention_cases import FORMS, short, split, whole
from gpu_util import bf16_dev, bits_host, say, to_dev

pytestmark = pytest.mark.gpu
FMT = {"bf16": w4.W4_KV_BF16, "e4m3": w4.W4_KV_E4M3, "q4": w4.W4_KV_Q4}


def check(case, seqs, heads):
    out, lse = w4.kv_attention(bf16_dev(case.q), to_dev(case.cache()), FMT[case.form], case.page, case.kv_heads,
                               to_dev(case.table), to_dev(case.lens), case.scale, case.window)
    torch.cuda.synchronize()
    got = oracle.bf16_bits_to_f64(bits_host(out))
    assert np.isfinite(got).all()
    lse = lse.cpu().numpy().astype(np.float64)
    for i in seqs:
        for h in heads:
            ref, rlse, bound, lb, _, _ = case.reference(i, h)
            err = np.abs(got[i, h] - ref)
            assert (err <= bound).all(), (i, h, np.max(err / bound))
            assert abs(lse[i, h] - rlse) <= lb, (i, h, lse[i, h], rlse, lb)


@pytest.mark.parametrize("form,D,group", FORMS)
@pytest.mark.parametrize("window", [0, 2500])
def test_whole_rows(form, D, group, window):
    say("[attn long] %s D=%d group=%d window=%d" % (form, D, group, window))
    case = whole(form, D, group, window)
    check(case, [0, 1, 2, 3, 4, 5, 6, 7, len(case.lens) - 1], [0, group - 1, 3 * group, 8 * group - 1])


@pytest.mark.parametrize("form,D,group", FORMS)
def test_split_rows(form, D, group):
    say("[attn long] %s D=%d group=%d split" % (form, D, group))
    check(split(form, D, group), [0, 1, 2], [0, 31 * group + group // 2, 64 * group - 1])


@pytest.mark.parametrize("form,D,group", FORMS)
@pytest.mark.parametrize("page", [16, 64])
def test_short_rows(form, D, group, page):
    say("[attn short] %s D=%d group=%d page=%d" % (form, D, group, page))
    case = short(form, D, group, page)
    check(case, range(len(case.lens)), range(case.heads))
