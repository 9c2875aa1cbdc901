"""CPU checks of the rules that cut calls into work: the sizes that GPU tests run take the forms that they are there for."""
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
