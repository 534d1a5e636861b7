"""The host's choice of decode kernels, from the sources: its functions are cut out of
csrc/dilattn.cu, with the constants of csrc/decode.cuh, and compiled into a host program."""
import functools
import os
import re
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_long_sequence_dilated_b200", "csrc")


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
    source = "#include <cstdio>\n" + "".join(f"constexpr int {n} = {v};\n" for n, v in constants().items()) \
        + _cut(host, "int decode_group(") + r"""
int main() {
  long long items;
  int lanes;
  while (std::scanf("%lld %d", &items, &lanes) == 2) std::printf("%d\n", decode_group(items, lanes));
}
"""
    folder = tempfile.mkdtemp(prefix="decode_route_")
    src, exe = os.path.join(folder, "route.cpp"), os.path.join(folder, "route")
    with open(src, "w", encoding="utf-8") as f:
        f.write(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", exe, src], check=True, capture_output=True, text=True)
    return exe


def ask(lines):
    """The program's numbers for each line of numbers."""
    text = "\n".join(" ".join(str(x) for x in line) for line in lines) + "\n"
    got = subprocess.run([program()], input=text, capture_output=True, text=True, check=True).stdout
    return [[int(x) for x in line.split()] for line in got.splitlines()]
