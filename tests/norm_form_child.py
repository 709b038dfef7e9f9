"""Child process of test_gpu_norm_forms.py: group norms under the form that the
parent asks for by ACP_NORM_FORM (the library reads it once per process), each
checked against binary64.  Prints one line a case and "all ok" at the end."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from tests.test_gpu_norm import PART_SHAPES, ROW_SHAPES, SHAPES, WIDE_SHAPES, Case  # noqa: E402


def main():
    form = {"slab": "slab", "parts": "by parts"}[os.environ["ACP_NORM_FORM"]]
    met = 0
    for k, (shape, groups) in enumerate(SHAPES + ROW_SHAPES + WIDE_SHAPES + PART_SHAPES[:4]):
        for dtype in ("f16", "bf16", "f32"):
            fmt = (None, "i8", "e4m3")[(k + len(dtype)) % 3]
            f, b = Case(shape, groups, dtype, ("silu", "none", "gelu")[k % 3], seed=k, fmt=fmt,
                        block=(32, 64, 128, 256)[k % 4]).run()
            assert "per row" not in f + b
            met += (form in f) + (form in b)
    assert met > 100, met
    print("all ok", flush=True)


if __name__ == "__main__":
    main()
