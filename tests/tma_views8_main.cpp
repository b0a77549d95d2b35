// Prints the TMA views of the int8 x int8 products (E n K on the command line), in the
// format of tma_views_main.cpp.  Built with the host compiler, no driver call.
#include <cstdio>
#include <cstdlib>

#include "tmap.cuh"

using moe::tmap::View;

static void print(const char* name, bool ok, const View& v) {
    if (!ok) {
        std::printf("%s refused\n", name);
        return;
    }
    std::printf("%s %d %d", name, v.rank, v.elem_bytes);
    for (int d = 0; d < v.rank; ++d) std::printf(" %llu", static_cast<unsigned long long>(v.dims[d]));
    for (int d = 0; d + 1 < v.rank; ++d) std::printf(" %llu", static_cast<unsigned long long>(v.strides[d]));
    for (int d = 0; d < v.rank; ++d) std::printf(" %u", static_cast<unsigned>(v.box[d]));
    std::printf("\n");
}

int main(int argc, char** argv) {
    if (argc != 4) return 2;
    const int E = std::atoi(argv[1]), n = std::atoi(argv[2]), K = std::atoi(argv[3]);
    View v;
    print("rows", moe::tmap::matrix8_view(&v, E * 7, K, 16, K), v);
    for (int c = 0; c < 2; ++c) {
        print(c ? "pairs_chunked" : "pairs", moe::tmap::pairs8_view(&v, E, n, K, 64, c != 0), v);
        print(c ? "quads_chunked" : "quads", moe::tmap::quads8_view(&v, E, n, K, c != 0), v);
    }
    return 0;
}
