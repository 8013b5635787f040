"""The numbers that the products keep for each device, compiled alone with fake lookups."""
import os
import subprocess

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "relative_bias_hybrid_gb300", "csrc",
                      "device_table.h")


def test_each_device_is_asked_for_itself(tmp_path):
    """One device's cluster count must not size the grids of another; a failed lookup (0) is
    not kept, and devices beyond the table are asked every time."""
    src, exe = tmp_path / "table.cpp", tmp_path / "table"
    src.write_text(f'''
#include "{HEADER}"
#include <cstdio>
static int calls = 0;
int main() {{
    inkattn::DeviceTable<2, 3> t;
    auto gives = [](int v) {{ return [v] {{ ++calls; return v; }}; }};
    if (t.get(0, 0, gives(76)) != 76 || t.get(1, 0, gives(74)) != 74) return 1;
    if (t.get(0, 0, gives(1)) != 76 || t.get(1, 0, gives(1)) != 74 || calls != 2) return 2;
    if (t.get(0, 1, gives(0)) != 0 || t.get(0, 1, gives(38)) != 38 || t.get(0, 1, gives(1)) != 38 || calls != 4) return 3;
    if (t.get(2, 0, gives(5)) != 5 || t.get(2, 0, gives(6)) != 6 || t.get(-1, 0, gives(7)) != 7 || calls != 7) return 4;
    std::puts("ok");
    return 0;
}}
''')
    subprocess.run(["g++", "-std=c++17", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.returncode


def test_the_products_keep_nothing_for_all_devices():
    """linear.cu holds what it asked of the runtime in that table and in no other static."""
    import re
    text = open(os.path.join(os.path.dirname(HEADER), "linear.cu")).read()
    assert re.findall(r"static (?!_assert|constexpr)[^;(]*", text) == ["static DeviceTable<64, 3> table"]
