#!/bin/bash
# Builds libemb.so (gfx950) from the HIP/C++ sources in this directory, the sources
# side by side.
set -euo pipefail
here="$(cd "$(dirname "${BASH_SOURCE[0]}")" && pwd)"
root="$(cd "$here/../.." && pwd)"
out="${1:-$here/../libemb.so}"
tmp="$out.tmp$$"
obj="$(mktemp -d)"
trap 'rm -rf "$obj"' EXIT
jobs=()
for src in plan.cpp forward.hip backward.hip table.hip noalloc.hip copy.hip attention.hip recurrence.hip delta.hip norm.hip rotary.hip; do
    hipcc --offload-arch=gfx950 -O3 -std=c++17 -fPIC \
        -Xclang -target-feature -Xclang -packed-fp32-ops \
        -Wall -Wno-unused-function \
        -I"$root/include" -I"$here" \
        -c "$here/$src" -o "$obj/$src.o" &
    jobs+=($!)
done
for job in "${jobs[@]}"; do wait "$job"; done
hipcc --offload-arch=gfx950 -fPIC -shared "$obj"/*.o -o "$tmp"
mv -f "$tmp" "$out"
