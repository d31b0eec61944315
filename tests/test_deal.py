"""csrc/deal.hpp compiled for the host: every unit of work is dealt to one
workgroup, whatever their number (no GPU needed)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_bf16_gemm_amd", "csrc")


def run(tmp_path, body):
    """Output lines of a host program with `body` as its main; nothing printed means nothing is wrong."""
    src = tmp_path / "check.cpp"
    src.write_text("#include <algorithm>\n#include <cstdio>\n#include <vector>\n"
                   "#define __host__\n#define __device__\n#define __forceinline__ inline\n"
                   '#include "deal.hpp"\nusing namespace gc;\n' f"int main() {{\n{body}\nreturn 0;\n}}\n")
    exe = tmp_path / "check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-500:]
    return r.stdout.splitlines()


@pytest.mark.parametrize("hand", [1, 5, 64])
def test_shares_cover_every_unit_once(tmp_path, hand):
    assert run(tmp_path, f"""
        const int hand = {hand};
        for (int G = 1; G <= 320; ++G)
            for (int units : {{0, 1, 7, 8, 63, 64, 65, 500, 1000, 2049}}) {{
                std::vector<int> taken(units);
                for (int b = 0; b < G; ++b) {{
                    Share s(b, G);
                    for (int u; (u = s.draw(hand, units)) >= 0;)
                        ++taken[u];
                }}
                if (std::count(taken.begin(), taken.end(), 1) != units)
                    printf("G %d units %d\\n", G, units);
            }}""") == []
