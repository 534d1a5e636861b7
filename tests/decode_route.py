"""The host's choice of decode kernels, from the sources, and the calls whose choice the tests pin.

The functions are cut out of csrc/dilattn.cu and csrc/decode.cuh, with the latter's constants, and
compiled into a host program. CASES are the calls that tests on the GPU make for the sake of one
route; a test on the CPU checks that each still takes it."""
import functools
import os
import re
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_long_sequence_dilated_b200", "csrc")
FIELDS = ("team", "dense", "grouped", "walks", "heads", "tokens", "nsub", "items", "group", "lanes", "warps",
          "plan_alone", "join_items")

DENSE = [(1 << 20, 1)]
PATS = {
    "dense": DENSE,
    "spread": [(1 << 20, 2), (1 << 20, 3), (8192, 1)],              # r that do not divide one another
    "nested": [(512, 1), (2048, 2), (8192, 4), (16384, 8)],
    "uneven": [(500, 1), (1200, 3), (6000, 6), (3330, 4)],
    "no_r1": [(600, 2), (1000, 3), (4000, 12)],                     # some tokens are kept by no pattern
    "sixteen": [(700 + 331 * i, r) for i, r in
                enumerate((5, 1, 2, 3, 4, 6, 20, 7, 8, 9, 10, 12, 14, 15, 18, 16))],
}
LAYOUTS = [(1, 1), (4, 2), (4, 1), (7, 1), (16, 1), (40, 1)]        # query heads, KV heads: 1 to 16 columns, and more
WIDE = 1200 * 16                                                   # positions of a table that teams are not given


def sub_items(H, Hkv):
    """Items of one token: its KV heads, more where one has over 16 query heads."""
    return Hkv * -(-(H // Hkv) // 16)


def copies(tokens, H, Hkv, items=260):
    """How often so many tokens have to come for this number of items: more than any team takes
    (128 or 256 blocks) of more than 16 tiles each."""
    return -(-items // (tokens * sub_items(H, Hkv)))


def _cases():
    got = {}

    def add(name, want, T, B, H, Hkv, d, pats, longest=WIDE, of_seq=True):
        got[name] = dict(T=T, B=B, H=H, Hkv=Hkv, d=d, pats=pats, longest=longest, of_seq=of_seq, want=want)

    for d in (64, 128):
        for H, Hkv in LAYOUTS:
            heads = {1: 1, 2: 2, 4: 4, 7: 8, 16: 16, 40: 16}[H // Hkv]
            add(f"few-spread-{H}-{Hkv}-{d}", dict(team=-1, heads=heads, join_items=1, grouped=0), 7, 7, H, Hkv, d,
                PATS["spread"])
            add(f"few-dense-{H}-{Hkv}-{d}", dict(team=-1, heads=heads, join_items=1, grouped=0, dense=1), 7, 7, H, Hkv,
                d, DENSE)
            for name in ("nested", "uneven", "no_r1", "sixteen"):
                add(f"many-{name}-{H}-{Hkv}-{d}",
                    dict(team=-1, heads=heads, grouped=0, lanes=16 if name == "sixteen" else 4),
                    7 * copies(7, H, Hkv), 7, H, Hkv, d, PATS[name])
            add(f"team-sixteen-{H}-{Hkv}-{d}", dict(heads=heads, lanes=16), 7, 7, H, Hkv, d, PATS["sixteen"])
        for name in ("dense", "spread"):
            for H, Hkv in ((1, 1), (4, 1)):
                add(f"long-{name}-{H}-{Hkv}-{d}", dict(team=-1, join_items=1, plan_alone=1), 2, 2, H, Hkv, d, PATS[name],
                    longest=70016, of_seq=False)
                add(f"long_among-{name}-{H}-{Hkv}-{d}", dict(team=-1, join_items=0), 320, 320, H, Hkv, d, PATS[name],
                    longest=40000, of_seq=False)
        # tokens of a sequence are taken together from one and a half a sequence on, padded slots or not
        for T, grouped in ((32, 0), (33, 0), (47, 0), (48, 1), (128, 1)):
            add(f"padded-{T}-{d}", dict(team=-1, grouped=grouped), T, 32, 8, 2, d, DENSE)
        # one workspace, used again and again: three tokens, and some hundred
        add(f"again-dense-3-{d}", dict(team=-1, grouped=0, dense=1, join_items=1), 3, 3, 8, 2, d, DENSE)
        add(f"again-spread-3-{d}", dict(team=-1, join_items=1), 3, 3, 8, 2, d, PATS["spread"])
        add(f"again-nested-200-{d}", dict(team=-1, join_items=0), 200, 3, 8, 2, d, PATS["nested"])
        add(f"again-drafts-12-{d}", dict(team=-1, grouped=1), 12, 3, 8, 2, d, DENSE)
        add(f"again-drafts-200-{d}", dict(team=-1, grouped=1), 200, 3, 8, 2, d, DENSE)
    return got


CASES = _cases()


def case(prefix):
    """Names of the cases that begin with this."""
    return [n for n in CASES if n.startswith(prefix)]


def _cut(text, head):
    """The definition that starts at `head`, through its matching closing brace."""
    i = text.index(head)
    depth, j = 0, text.index("{", i)
    for k in range(j, len(text)):
        depth += (text[k] == "{") - (text[k] == "}")
        if depth == 0:
            return text[i:k + 1]
    raise ValueError(head)


def constants():
    """The integer constants of decode.cuh, by name."""
    text = open(os.path.join(CSRC, "decode.cuh"), encoding="utf-8").read()
    got = {}
    for line in re.findall(r"^constexpr int (k.*?);", text, re.M):
        for part in line.split(","):
            name, value = part.split("=")
            got[name.strip()] = eval(value, {}, got)
    return got


@functools.lru_cache(maxsize=None)
def program():
    """The compiled program: lines in, a line of numbers out for each."""
    host = open(os.path.join(CSRC, "dilattn.cu"), encoding="utf-8").read()
    device = open(os.path.join(CSRC, "decode.cuh"), encoding="utf-8").read()
    heads = ("int decode_heads(", "int decode_tokens(", "int decode_columns(", "long long decode_items(",
             "int decode_team(", "int decode_group(", "struct DecodeRoute {", "DecodeRoute decode_route(")
    source = "#include <algorithm>\n#include <cstdio>\n" \
        + "".join(f"constexpr int {n} = {v};\n" for n, v in constants().items()) \
        + _cut(device, "constexpr int decode_blocks_per_sm(") + "\n" \
        + "\n".join(_cut(host, h) + (";" if h.startswith("struct") else "") for h in heads) + r"""
int main() {
  char what;
  while (std::scanf(" %c", &what) == 1) {
    if (what == 'g') {
      long long items;
      int lanes;
      if (std::scanf("%lld %d", &items, &lanes) != 2) return 1;
      std::printf("%d\n", decode_group(items, lanes));
    } else {
      int T, B, Hkv, G, d, of_seq, sms, npat, w[16], r[16];
      long long longest;
      if (std::scanf("%d %d %d %d %d %d %lld %d %d", &T, &B, &Hkv, &G, &d, &of_seq, &longest, &sms, &npat) != 9) return 1;
      for (int i = 0; i < npat; ++i)
        if (std::scanf("%d %d", &w[i], &r[i]) != 2) return 1;
      const DecodeRoute a = decode_route(T, B, Hkv, G, d, of_seq != 0, w, r, npat, longest, sms);
      std::printf("%d %d %d %d %d %d %d %d %d %d %d %d %d\n", a.team, a.dense, a.grouped, a.walks, a.heads, a.tokens,
                  a.nsub, a.items, a.group, a.lanes, a.warps, a.plan_alone, a.join_items);
    }
  }
}
"""
    folder = tempfile.mkdtemp(prefix="decode_route_")
    src, exe = os.path.join(folder, "route.cpp"), os.path.join(folder, "route")
    with open(src, "w", encoding="utf-8") as f:
        f.write(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", exe, src], check=True, capture_output=True, text=True)
    return exe


def _ask(lines):
    text = "\n".join(" ".join(str(x) for x in line) for line in lines) + "\n"
    got = subprocess.run([program()], input=text, capture_output=True, text=True, check=True).stdout
    return [[int(x) for x in line.split()] for line in got.splitlines()]


def groups(pairs):
    """The items of a group for each (items, threads to an item)."""
    return [g for g, in _ask([("g", n, lanes) for n, lanes in pairs])]


def routes(calls, sms=148):
    """The route of each call (a dict as in CASES), as a dict of FIELDS."""
    got = _ask([("r", c["T"], c["B"], c["Hkv"], c["H"] // c["Hkv"], c["d"], int(c["of_seq"]), c["longest"], sms,
                 len(c["pats"]), *(x for p in c["pats"] for x in p)) for c in calls])
    return [dict(zip(FIELDS, g)) for g in got]
