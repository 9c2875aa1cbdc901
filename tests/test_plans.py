"""CPU checks of the rules that cut calls into work: the sizes that GPU tests run take the forms that they are there for."""
import math
import random

from qlora_linear_layers_nf4_b200 import nf4qlora as Q
from tests import test_fp8_forms_gpu as fp8
from tests import test_gated_forms_gpu as forms
from tests.plans import SMS, ask


def test_decode_cases_take_their_splits():
    plans = ask(*[("decode", m, n, k, SMS) for m, n, k, *_ in forms.DECODE])
    streams = ask(*[("streams", m, n, k, r, SMS) for m, n, k, r, *_ in forms.DECODE])
    for case, p, s in zip(forms.DECODE, plans, streams):
        kind = "none" if p["rest"] == 0 else "own" if p["rest_ctas"] % p["rest"] == 0 and p["rest_ctas"] > p["rest"] else "straddle"
        assert s["streams"] and (p["whole"], kind) == case[-2:], (case, p)


def test_few_tokens_of_the_gemm():
    cases = forms.FEW_BY_GEMM
    assert not any(p["streams"] for p in ask(*[("streams", m, n, k, r, SMS) for m, n, k, r, _ in cases]))
    plans = ask(*[("gemm", 0, m, n, k, r, SMS) for m, n, k, r, _ in cases])
    assert any(p["splits"] > 1 for p in plans) and any(p["splits"] == 1 for p in plans)


def test_two_mma_cases_take_two():
    for backward, cases in ((0, forms.TWO_MMAS_FWD), (1, forms.TWO_MMAS_DX)):
        plans = ask(*[("gemm", backward, m, n, k, r, SMS) for m, n, k, r, *_ in cases])
        assert all(p["parts"] == 2 for p in plans), plans
        # one of them ends with a token tile of a single part, one has more tiles than CTA pairs
        assert any(0 < m - (p["row_tiles"] - 1) * p["tile_rows"] <= 256 < p["tile_rows"] for (m, *_), p in zip(cases, plans))
        assert any(p["tiles"] > p["pairs"] for p in plans)


def test_split_cases_take_several_rounds():
    for (m, n, k, r, _), p in zip(forms.ROUNDS_OF_SPLITS, ask(*[("gemm", 0, m, n, k, r, SMS) for m, n, k, r, _ in forms.ROUNDS_OF_SPLITS])):
        assert p["splits"] > 1 and p["tiles"] > 2 * p["pairs"], ((m, n, k, r), p)


def test_streamed_8_bit_cases_take_several_rounds():
    for (m, n, k, *_, rounds), p in zip(fp8.STREAMED, ask(*[("fp8", m, n, k, SMS) for m, n, k, *_ in fp8.STREAMED])):
        assert p["streams"] and -(-p["groups"] // p["ctas"]) == rounds, ((m, n, k), p)


# n, k, us of a forward of 24 tokens (r = 16) by streaming the weights and by the GEMM, measured on 148 SMs
GATED_24 = [
    (11008, 4096, 47.2, 53.0), (14336, 4096, 58.4, 63.0), (20480, 5120, 94.6, 103.8), (28672, 8192, 204.0, 223.6),
    (1000, 4096, 15.0, 16.7), (1024, 1024, 11.1, 14.7), (1024, 8192, 19.1, 27.3), (512, 512, 10.4, 11.5), (5504, 4096, 27.8, 32.2),
    (2752, 4096, 24.4, 21.9), (4096, 4096, 28.6, 25.9), (8192, 2048, 25.0, 23.5), (4096, 512, 15.3, 11.6), (4096, 1024, 16.2, 16.4),
    (4736, 512, 9.1, 11.9), (8192, 1024, 18.1, 16.7), (11008, 1024, 22.4, 24.6), (1536, 1536, 13.5, 14.5), (200, 2048, 12.4, 14.5),
    (4096, 2048, 18.9, 18.6), (6144, 2048, 20.2, 23.4), (7040, 2048, 20.9, 23.4), (2560, 2560, 21.9, 18.4), (2368, 4096, 18.8, 21.8),
    (3584, 4096, 25.7, 24.4), (4736, 4096, 23.9, 32.4), (4800, 4096, 26.5, 32.2), (6144, 4096, 29.9, 38.1), (7040, 4096, 32.9, 37.7),
    (7168, 4096, 35.4, 37.6), (8192, 4096, 38.9, 37.8), (9216, 4096, 41.6, 43.6), (9472, 4096, 40.0, 44.0), (12032, 4096, 51.5, 53.0),
    (14208, 4096, 55.8, 62.3), (16384, 4096, 65.2, 66.5), (17920, 4096, 71.6, 66.5), (18944, 4096, 72.0, 72.7), (24576, 4096, 92.4, 94.9),
    (5120, 5120, 31.4, 35.8), (13824, 5120, 69.0, 73.6), (3000, 8192, 35.7, 39.3), (8192, 8192, 67.4, 70.7), (22016, 8192, 159.7, 168.5),
    (9216, 2048, 27.3, 28.9), (17920, 2048, 42.5, 38.1), (18000, 2048, 42.7, 42.4), (4096, 3584, 25.8, 25.2), (8448, 4096, 39.3, 37.5),
    (8960, 4096, 41.1, 42.9), (2560, 5120, 26.4, 25.5), (4096, 5120, 32.2, 29.8), (7168, 5120, 40.9, 45.5), (8192, 5120, 44.6, 45.7),
    (9216, 5120, 49.4, 51.1), (17920, 5120, 86.5, 81.5), (3000, 6144, 29.5, 33.7), (4096, 6144, 34.8, 34.6), (3000, 7168, 32.0, 37.7),
    (2752, 8192, 34.1, 32.8), (4096, 8192, 41.3, 41.8), (7168, 8192, 59.5, 63.7), (9216, 8192, 74.9, 76.0), (2560, 10240, 36.9, 38.1),
]


def test_the_faster_kernel_takes_17_to_32_tokens():
    """Within 7 %; and the rule is the same for every count of tokens from 17 to 32, and up to 16."""
    for m in (17, 24, 32):
        for (n, k, stream, gemm), p in zip(GATED_24, ask(*[("streams", m, n, k, 16, SMS) for n, k, *_ in GATED_24])):
            assert (stream if p["streams"] else gemm) <= 1.07 * min(stream, gemm), (m, n, k, p)
    assert all(p["streams"] for p in ask(*[("streams", m, n, k, 16, SMS) for m in (1, 8, 16) for n, k, *_ in GATED_24]))
    assert not any(p["streams"] for p in ask(*[("streams", 33, n, k, 16, SMS) for n, k, *_ in GATED_24]))


# n, k, then (tokens, us of the few-token kernel, us of the tensor-core kernel), codes given, measured on 148 SMs
FP8_FEW = [
    (4096, 4096, (1, 6.4, 8.4), (4, 7.0, 8.9), (8, 7.6, 9.0)),
    (11008, 4096, (1, 11.9, 13.5), (4, 12.7, 13.9), (8, 12.6, 13.4)),
    (14336, 4096, (1, 13.9, 14.9), (4, 14.5, 15.0), (8, 14.9, 14.6)),
    (32000, 4096, (1, 25.9, 27.0), (4, 26.3, 26.8), (8, 27.1, 26.5)),
    (2048, 2048, (1, 3.9, 6.5), (4, 4.3, 6.4), (8, 4.1, 6.0)),
    (512, 512, (1, 2.4, 3.5), (4, 2.4, 3.4), (8, 2.5, 3.5)),
    (1000, 2064, (1, 3.0, 5.5), (4, 3.3, 5.4), (8, 3.4, 5.6)),
    (1024, 5120, (1, 5.4, 6.7), (4, 6.0, 7.1), (8, 6.7, 7.2)),
    (4096, 5120, (1, 7.8, 9.0), (4, 8.6, 9.5), (8, 9.3, 9.7)),
    (8192, 5120, (1, 12.8, 12.7), (4, 13.0, 13.0), (8, 13.7, 12.9)),
    (11008, 5120, (1, 14.9, 15.2), (4, 15.6, 15.5), (8, 16.3, 15.5)),
    (16384, 5120, (1, 21.2, 18.3), (4, 21.7, 18.3), (8, 22.7, 18.2)),
    (24576, 5120, (1, 27.1, 30.7), (4, 28.0, 31.3), (8, 29.5, 30.7)),
    (1024, 8192, (1, 6.9, 7.9), (4, 7.2, 8.0), (8, 8.1, 8.0)),
    (4096, 8192, (1, 10.2, 11.7), (4, 10.5, 11.8), (8, 11.3, 12.0)),
    (8192, 8192, (1, 15.6, 16.7), (4, 16.7, 16.9), (8, 17.6, 17.3)),
    (11008, 8192, (1, 20.0, 22.4), (4, 20.6, 22.5), (8, 22.8, 22.7)),
    (16384, 8192, (1, 26.6, 28.3), (4, 28.0, 27.4), (8, 29.7, 26.9)),
    (28672, 8192, (1, 40.1, 47.3), (4, 41.3, 49.3), (8, 43.9, 49.4)),
    (1024, 11008, (1, 8.6, 9.0), (4, 9.5, 8.9), (8, 10.8, 8.8)),
    (4096, 11008, (1, 11.9, 13.3), (4, 13.2, 13.4), (8, 15.1, 13.1)),
    (8192, 11008, (1, 21.4, 20.6), (4, 23.1, 20.9), (8, 25.7, 20.9)),
    (16384, 11008, (1, 35.6, 36.5), (4, 37.0, 36.5), (8, 41.3, 35.2)),
    (24576, 11008, (1, 47.8, 64.7), (4, 50.0, 61.6), (8, 55.2, 61.7)),
    (1024, 14336, (1, 10.6, 9.2), (4, 11.8, 9.6), (6, 12.5, 9.6)),
    (4096, 14336, (1, 13.9, 15.5), (4, 15.7, 15.6), (6, 17.5, 15.5)),
    (8192, 14336, (1, 25.5, 24.5), (4, 28.1, 24.9), (6, 30.0, 24.9)),
    (16384, 14336, (1, 44.6, 42.7), (4, 46.7, 49.5), (6, 50.2, 42.7)),
    (24576, 14336, (1, 59.8, 76.1), (4, 62.7, 76.3), (6, 67.4, 78.5)),
    (2048, 28672, (1, 19.1, 18.8), (3, 20.2, 18.5)),
    (4096, 28672, (1, 25.0, 24.9), (3, 28.0, 24.8)),
    (8192, 28672, (1, 44.0, 43.1), (3, 48.7, 45.3)),
]
# n, k, then (tokens, us of a whole call that quantizes them in every CTA, and with a launch of its own for that)
FP8_INSIDE = [
    (512, 512, (1, 2.5, 4.1), (2, 2.6, 4.6), (3, 2.8, 4.6), (4, 2.8, 4.3), (5, 2.9, 4.4), (6, 3.0, 4.6), (7, 3.0, 4.4), (8, 3.0, 4.5)),
    (512, 2048, (1, 3.1, 4.4), (2, 3.5, 4.6), (3, 4.3, 5.0), (4, 4.9, 5.1)),
    (512, 4096, (1, 4.4, 5.6), (2, 5.7, 6.0)),
    (512, 8192, (1, 8.6, 9.2)),
    (1000, 2064, (1, 3.6, 4.9), (2, 4.2, 5.5), (3, 4.7, 5.3)),
    (1024, 1024, (1, 2.6, 4.1), (2, 2.8, 4.7), (3, 3.1, 4.3), (4, 3.1, 4.8), (6, 4.2, 5.1), (8, 4.4, 5.0)),
    (1024, 2048, (1, 3.4, 4.8), (2, 3.8, 5.0), (3, 4.6, 5.3), (4, 5.1, 5.3)),
    (1024, 4096, (1, 5.6, 6.8), (2, 6.7, 7.3)),
    (1024, 8192, (1, 8.7, 9.4)),
    (2048, 1024, (1, 2.7, 4.7), (2, 2.9, 4.4), (3, 3.2, 4.8), (4, 3.3, 4.6), (6, 4.3, 5.0), (8, 4.8, 5.1)),
    (2048, 2048, (1, 4.6, 6.2), (2, 4.9, 6.2), (3, 5.7, 6.5), (4, 6.0, 6.7)),
    (2048, 4096, (1, 6.0, 7.5), (2, 7.2, 7.6)),
    (2048, 5632, (1, 8.2, 9.2)),
    (2048, 8192, (1, 9.7, 10.4)),
    (4096, 1024, (1, 4.3, 5.9), (2, 4.6, 5.8), (3, 4.4, 5.4), (4, 4.7, 5.5), (6, 6.1, 6.3), (8, 6.5, 6.5)),
    (4096, 2048, (1, 5.5, 7.2), (2, 5.5, 6.5), (3, 6.8, 7.5), (4, 7.4, 7.5)),
    (4096, 4096, (1, 7.7, 8.4), (2, 9.1, 8.6)),
    (4096, 5632, (1, 10.0, 10.1)),
    (4096, 8192, (1, 12.1, 12.7)),
    (5632, 2048, (1, 7.2, 8.3), (2, 7.6, 8.4), (3, 8.7, 8.8), (4, 8.9, 8.1)),
    (8192, 1024, (1, 5.9, 7.5), (2, 6.2, 7.3), (3, 6.3, 7.7), (4, 6.5, 7.5), (6, 7.7, 7.7), (8, 8.1, 8.0)),
    (8192, 2048, (1, 8.0, 9.3), (2, 8.3, 9.3), (3, 9.4, 9.7), (4, 9.9, 9.7)),
    (8192, 4096, (1, 12.0, 12.6), (2, 13.2, 13.0)),
    (8192, 8192, (1, 18.0, 18.5)),
    (11008, 1024, (1, 6.9, 8.4), (2, 7.2, 8.6), (3, 7.5, 8.6), (4, 7.9, 7.9), (6, 8.7, 8.0), (8, 9.1, 8.3)),
    (11008, 2048, (1, 9.7, 10.8), (2, 10.1, 10.8), (3, 10.9, 11.2), (4, 11.4, 11.1)),
    (11008, 4096, (1, 13.8, 13.6), (2, 15.3, 14.3)),
    (14336, 4096, (1, 17.3, 16.4), (2, 18.0, 16.3)),
    (16384, 1024, (1, 8.9, 10.2), (2, 9.1, 9.9), (3, 9.5, 10.3), (4, 9.6, 10.2), (6, 10.9, 10.5), (8, 11.1, 10.5)),
    (16384, 2048, (1, 12.5, 13.0), (2, 12.6, 12.9), (3, 13.5, 13.4), (4, 14.0, 13.5)),
    (16384, 4096, (1, 18.6, 17.7), (2, 19.9, 18.6)),
    (28672, 8192, (1, 44.8, 41.6)),
    (32000, 1024, (1, 13.7, 13.9), (2, 13.9, 13.8), (3, 14.5, 14.1), (4, 14.6, 14.0), (6, 15.7, 14.6), (8, 16.4, 14.5)),
    (32000, 2048, (1, 18.9, 18.7), (2, 19.4, 18.9), (3, 20.3, 19.3), (4, 20.8, 19.2)),
    (32000, 4096, (1, 29.7, 27.0), (2, 31.2, 28.4)),
]


def test_the_faster_8_bit_kernel_takes_few_tokens():
    """Within 11 %."""
    cases = [(m, n, k, a, b) for n, k, *times in FP8_FEW for m, a, b in times]
    for (m, n, k, few, tensor), p in zip(cases, ask(*[("fp8", m, n, k, SMS) for m, n, k, *_ in cases])):
        assert (few if p["streams"] else tensor) <= 1.11 * min(few, tensor), (m, n, k, p)
    cases = [(m, n, k, a, b) for n, k, *times in FP8_INSIDE for m, a, b in times]
    for (m, n, k, inside, before), p in zip(cases, ask(*[("fp8", m, n, k, SMS) for m, n, k, *_ in cases])):
        if p["streams"]:
            assert (inside if p["inside"] else before) <= 1.11 * min(inside, before), (m, n, k, p)


def test_splits_fit_their_workspace():
    """On devices of any number of SMs; and batches that always stream their weights have no room for splits."""
    rng = random.Random(7)
    cases = [(rng.randint(0, 1), round(math.exp(rng.uniform(0, 9))), 8 * round(math.exp(rng.uniform(0, 7.6))),
              64 * round(math.exp(rng.uniform(0, 5.2))), 8 * rng.randint(1, 32), rng.choice((16, 78, 132, 148, 160, 200))) for _ in range(20000)]
    plans = ask(*[("gemm", *c) for c in cases])
    room = ask(*[("bytes", *c[:5]) for c in cases])
    streams = ask(*[("streams", *c[1:]) for c in cases])
    split = 0
    for (back, m, n, k, r, _), p, b, s in zip(cases, plans, room, streams):
        if p["splits"] > 1 and (back or not s["streams"]):
            split += 1
            assert p["splits"] * m * (k if back else 2 * n) * 4 <= b["bytes"], (back, m, n, k, r, p)
    assert split > 1000
    for m in (1, 16):
        assert Q.workspace_bytes(Q.OP_GATED_FWD, m, 11008, 4096, 64, 64, True) < 4 << 20
    assert Q.workspace_bytes(Q.OP_GATED_FWD, 100, 11008, 1024, 64, 64, True) < 4 << 20   # too few steps to split
