"""The row of a dropout's block of eight values, at sizes that no GPU test reaches:
the function that the kernel calls, compiled for the host."""
import os
import random
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_of_blocks(tmp_path):
    from mixed_precision_adam_grad_gb300 import build
    exe = str(tmp_path / "dropout_rows")
    subprocess.run(["nvcc", "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, *build.ARCH,
                    os.path.join(ROOT, "tests", "c", "dropout_rows.cu"), "-o", exe], check=True)
    rng = random.Random(1)
    # blocks of a row on both sides of 32 bits; a tensor has 2^37 of them at most
    pairs = [(b, c) for c in (1, 3, 2 ** 31 - 1, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 33, 2 ** 36)
             for b in (0, 1, c - 1, c, c + 1, 2 * c - 1, 2 ** 32 - 1, 2 ** 32, 2 ** 37 - 1)]
    pairs += [(rng.randrange(1 << rng.randint(1, 37)), rng.randrange(1, 1 << rng.randint(1, 37))) for _ in range(2000)]
    r = subprocess.run([exe], input="\n".join("%d %d" % p for p in pairs), capture_output=True, text=True, check=True)
    assert [int(v) for v in r.stdout.split()] == [b // c for b, c in pairs]
