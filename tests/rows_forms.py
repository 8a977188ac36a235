"""Which work-group form the row-wise calls take for given sizes: the rules of rows_api.hip and
rows_plan.h over again, with the thresholds read from those sources, so that tests can choose
sizes by the form that they mean and see when a moved threshold takes them elsewhere."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "group_wise_bit_amd", "csrc", "rows")


def _find(name, pattern):
    found = re.findall(pattern, open(os.path.join(CSRC, name)).read())
    assert len(found) == 1, (name, pattern, found)
    return found[0]


def _constant(name, which):
    value = _find(name, rf"constexpr \w+ {which} = ([0-9 <]+);")
    return eval(value, {"__builtins__": {}})              # digits, spaces and << only


DIRECT_PAIRS = _constant("rows_api.hip", "kDirectPairs")
DIRECT_BYTES = _constant("rows_api.hip", "kDirectBytes")
TILED_ROWS = _constant("rows_api.hip", "kTiledRows")
SORT_RANKS = _constant("rows_api.hip", "kSortRanks")
DOT_RANK = _constant("rows.h", "kDotRank")
PLAN_IDS = _constant("group.h", "kPlanIds")
PLAN_GROUPS = _constant("group.h", "kPlanGroups")
KSPLIT_HALF = int(_find("rows_plan.h", r"c\.half = groups <= (\d+);"))
KSPLIT_WAVES = tuple(map(int, _find("rows_plan.h", r"c\.waves = groups < (\d+) \? (\d+) : (\d+);")))
GEMV_HALF = int(_find("rows_plan.h", r"c\.half = groups < (\d+);"))
GEMV_WAVES = tuple(map(int, _find("rows_plan.h", r"c\.waves = c\.half && items > (\d+) \? (\d+) : (\d+);")))
TILED_GROUPS = int(_find("rows_plan.h", r"\* tiles >= (\d+) &&"))


def tiles_of(n):
    return -(-n // 64)


def packed_bytes(n, k, bits):
    return tiles_of(n) * 64 * (k // 64) * 2 * bits * 4


def ksplit(groups):
    """(columns, waves) of the 32-row form."""
    return 32 if groups <= KSPLIT_HALF else 64, KSPLIT_WAVES[1 if groups < KSPLIT_WAVES[0] else 2]


def gemv(items, groups):
    """(columns, waves) of the one-row form."""
    half = groups < GEMV_HALF
    return 8 if half else 16, GEMV_WAVES[1 if half and items > GEMV_WAVES[0] else 2]


def tiled(cols, tiles, m, ld, k):
    return cols * tiles >= TILED_GROUPS and ((m - 1) * ld + k) * 2 < 1 << 32


def moe(m, top_k, experts, inner, model, bits, dbits, ld=None):
    """(rows per work-group, form of gate and up, form of down)."""
    pairs, ki, km = m * top_k, inner // 64, model // 64
    if pairs <= DIRECT_PAIRS and pairs * (2 * packed_bytes(inner, model, bits) +
                                          packed_bytes(model, inner, dbits)) <= DIRECT_BYTES:
        return 1, gemv(km, pairs * 4 * ki), gemv(top_k * ki, m * 4 * km)
    if pairs >= TILED_ROWS * experts and \
            tiled((ki + 1) // 2, pairs // 64 + experts // 2, m, model if ld is None else ld, model):
        return 64, None, None
    used = min(pairs, experts)
    return 32, ksplit(ki * used), ksplit(km * used)


def lora(m, n, k, rank, ld=None):
    """(rows per work-group, how the adapters are added, form): by "dots" of the threads, on
    the matrix cores with the rows as they "come", or "ordered" by adapter."""
    is_tiled = tiled(-(-tiles_of(n) // 4), -(-m // 64), m, k if ld is None else ld, k)
    if is_tiled:
        return 64, "ordered", None
    how = "ordered" if m * rank >= SORT_RANKS else "dots" if rank <= DOT_RANK else "come"
    return 32, how, ksplit(tiles_of(n) * -(-m // 32))


def _align(b):
    return -(-b // 256) * 256


def _tile_bound(count, buckets, height):
    return count // height + min(count, buckets)


def _plan_bytes(count, buckets, height):
    b = _align(4 * count) + _align(16 * _tile_bound(count, buckets, height)) + _align(4)
    return b + (_align(4 * PLAN_GROUPS * (buckets + 1)) if count > PLAN_IDS else 0)


def moe_workspace(m, top_k, experts, inner, model, bits, dbits):
    """What qlin_moe_mlp_workspace_bytes gives if the form is the one above."""
    pairs = m * top_k
    b = 65536 + _align(4 * pairs * inner)
    if moe(m, top_k, experts, inner, model, bits, dbits)[0] != 1:
        b += _plan_bytes(pairs, experts, 32) + _align(4 * pairs * model)
    return b


def lora_workspace(m, n, k, slots, rank):
    """What qlin_gemm_lora_workspace_bytes gives if the form is the one above."""
    rp, splits, b = -(-rank // 16) * 16, 1, 65536
    if lora(m, n, k, rank)[1] == "ordered":
        steps, tiles = -(-k // 128), _tile_bound(m, slots, 16)
        while splits < 8 and tiles * splits < 256 and steps >= 16 * splits:
            splits *= 2
        splits = -(-steps // -(-steps // splits))
        b += _plan_bytes(m, slots, 16)
    return b + _align(4 * splits * m * rp)
