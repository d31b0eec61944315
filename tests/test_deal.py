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


@pytest.mark.parametrize("groups,S,bm", [(1024, (1 << 27) - 1, 16), (1024, 1 << 26, 16), (1000, 3000, 64),
                                         (7, (1 << 27) - 1, 16), (1023, (1 << 27) - 1, 32)])
def test_tiles_of_falling_offsets_stay_in_their_groups(tmp_path, groups, S, bm):
    """Offsets 0, S, 0, S, ...: whatever the sum of the groups' tiles is, a tile's place in its group is
    one that the group has.  (The prefix sum of the kernels, by threads, waves and the workgroup.)"""
    assert run(tmp_path, f"""
        const int n = {groups}, S = {S}, bm = {bm}, threads = 256, per = 1024 / threads;
        auto count = [&](int e) {{ return e < n && e % 2 == 0 ? (S + bm - 1) / bm : 0; }};
        std::vector<int> first(n + 1), inc(threads), wave(threads / 64, 0);
        for (int t = 0; t < threads; ++t) {{
            int sum = 0;
            for (int i = 0; i < per; ++i)
                sum = add_tiles(sum, count(per * t + i));
            inc[t] = t % 64 ? add_tiles(inc[t - 1], sum) : sum;
            if (t % 64 == 63)
                wave[t / 64] = inc[t];
        }}
        int all = 0;
        for (int w : wave)
            all = add_tiles(all, w);
        for (int t = 0; t < threads; ++t) {{
            int before = 0;
            for (int w = 0; w < t / 64; ++w)
                before = add_tiles(before, wave[w]);
            int at = add_tiles(before, t % 64 ? inc[t - 1] : 0);
            for (int i = 0; i < per; ++i) {{
                if (per * t + i < n)
                    first[per * t + i] = at;
                at = add_tiles(at, count(per * t + i));
            }}
        }}
        first[n] = all;
        const int64_t real = (int64_t)(n + 1) / 2 * ((S + bm - 1) / bm);
        if (all != std::min<int64_t>(real, MOST_TILES))
            printf("sum %d\\n", all);
        for (int e = 0; e < n; ++e)
            if (first[e + 1] < first[e] || first[e + 1] - first[e] > count(e))
                printf("group %d from %d to %d\\n", e, first[e], first[e + 1]);""") == []


@pytest.mark.parametrize("per_tile", [1, 2, 3, 4, 5, 7, 8, 9, 56])
def test_line_is_cut_into_pieces(tmp_path, per_tile):
    """The pieces follow one another over the whole line, no tile is cut with fewer than `least` quads on a
    side, every quad is found in its piece, and tiles that are not worth cutting go to as many workgroups
    as there are."""
    assert run(tmp_path, f"""
        const int per = {per_tile};
        for (int G : {{1, 3, 64, 255, 256}})
            for (int tiles : {{1, 2, 5, 63, 128, 255, 256, 257, 448, 1000}})
                for (int smallest : {{4, per}}) {{
                    const Line l(tiles, per, smallest, G);
                    bool ok = l.pieces >= 1 && l.pieces <= G && l.bound(0) == 0 && l.bound(l.pieces) == (int64_t)tiles * per;
                    int64_t longest = 0;
                    for (int w = 0; w < l.pieces; ++w) {{
                        const int64_t a = l.bound(w), b = l.bound(w + 1);
                        const int r = (int)(b % per);
                        ok &= a <= b && (r == 0 || (r >= smallest && per - r >= smallest));
                        longest = std::max(longest, b - a);
                        for (int64_t q = a; q < b; ++q)
                            ok &= l.piece_of(q) == w;
                    }}
                    if (per <= smallest)
                        ok &= longest == (int64_t)(tiles + G - 1) / G * per;
                    if (!ok)
                        printf("G %d tiles %d smallest %d pieces %d longest %d\\n", G, tiles, smallest, l.pieces, (int)longest);
                }}""") == []


def test_pieces_of_sums_have_room(tmp_path):
    """However many compute units there are, all pieces' sums fit the workspace (one always does)."""
    assert run(tmp_path, """
        const int64_t room = (int64_t)64 << 20;
        for (int64_t cus : {1, 32, 256, 304, 1024, 4096})
            for (int64_t S : {1, 17, 64, 1000, 4096, 16384, 131072, 1 << 20})
                for (int r : {8, 64, 128})
                    for (int steps : {0, 7, 8, 64, 224, 4096})
                        for (int bm : {16, 64})
                            for (int64_t groups : {1, 8, 1000}) {
                                const int64_t plane = S * r * 4;
                                const int n = sum_pieces(cus, std::min(S, S / bm + groups), steps, plane, room);
                                if (n < 1 || n > 16 || (n > 1 && (n * plane > room || steps / n < 8)))
                                    printf("cus %d S %d r %d steps %d pieces %d\\n", (int)cus, (int)S, r, steps, n);
                            }""") == []


def test_adapter_cases_walk_their_loops(tmp_path):
    """The sizes of adapter_cases reach what they are there for: the span of rows or columns, and more
    units of work (with the rows of no adapter, which are copied) than workgroups."""
    from adapter_cases import COLUMNS, ROWS
    cases = [(c, True) for c in ROWS] + [(c, False) for c in COLUMNS]
    out = run(tmp_path, "ExpandPlan p;\n" + "\n".join(
        f'p = expand_plan({M}, {N}, {len(sizes)}, {r}, 256); printf("%d %d %d %d\\n", p.rows, p.span, p.spans, (int)p.grid);'
        for (M, K, N, r, sizes, span, again), _ in cases))
    for ((M, K, N, r, sizes, span, again), many), line in zip(cases, out):
        rows, got, spans, grid = map(int, line.split())
        height = got if many else 16
        units = sum(-(-n // height) for n in [*sizes, M - sum(sizes)]) * spans
        assert (rows, got, units > grid) == (many, span, again), (M, N, r, line, units)
        assert sum(sizes) < M
