// The launches of the feed-forward products, recorded on the CPU: the library's
// own host code (zero_ffn.hip, its host half) over a stub launch that keeps what
// a kernel would get. Built and run by test_ffn_launch.py, without a GPU; the
// operands are addresses that nothing reads.
#include <cstdio>
#include <cstdlib>

#include "zero_ffn.hip"

using namespace zero;

namespace {
dim3 grid, block;
size_t shared_bytes;
hipStream_t stream;

constexpr uint64_t kSpace = uint64_t{1} << 50;  // the workspace's address

template <class T, FfnKind KIND, bool FAST>
bool is(const void* f) { return f == reinterpret_cast<const void*>(&ffn_kernel<T, KIND, FAST>); }

template <FfnKind KIND>
const char* path(const void* f)
{
    if (is<Big<KIND>, KIND, true>(f) || is<Mid, KIND, true>(f)) return "direct";
    if constexpr (KIND != kFfnWeight)
        if (is<Small, KIND, true>(f) || is<Flat, KIND, true>(f)) return "direct";
    return is<Slow, KIND, false>(f) ? "registers" : nullptr;
}
}  // namespace

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t n, hipStream_t s)
{
    grid = g, block = b, shared_bytes = n, stream = s;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* n, hipStream_t* s)
{
    *g = grid, *b = block, *n = shared_bytes, *s = stream;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
// what a program with kernels calls at its start
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
// A line for each launch: what it is, then for a copy the operands (from, ld,
// rows, cols, to), for a product its factors as the kernel gets them (address
// and ld of d, d, h, w, w) and where its parts begin and end.
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3, void** args, size_t, hipStream_t)
{
    if (f == reinterpret_cast<const void*>(&ffn_copy_kernel)) {
        const CopyArgs& c = *static_cast<CopyArgs*>(args[0]);
        std::printf("copy");
        for (unsigned i = 0; i < g.y; ++i)
            std::printf(" %ld %ld %ld %ld %ld", reinterpret_cast<long>(c.from[i].p), static_cast<long>(c.from[i].ld), static_cast<long>(c.from[i].rows),
                        static_cast<long>(c.from[i].cols), reinterpret_cast<long>(c.to[i]));
        std::printf("\n");
        return hipSuccess;
    }
    const char* what = path<kFfnForward>(f);
    if (what == nullptr) what = path<kFfnInput>(f);
    if (what == nullptr) what = path<kFfnWeight>(f);
    if (what == nullptr) return hipSuccess;  // a join
    const FfnArgs& a = *static_cast<FfnArgs*>(args[0]);
    std::printf("%s", what);
    for (int i = 0; i < 2; ++i) std::printf(" %ld %ld", reinterpret_cast<long>(a.d[i]), static_cast<long>(a.ld_d[i]));
    std::printf(" %ld %ld", reinterpret_cast<long>(a.h), static_cast<long>(a.ld_h));
    for (int i = 0; i < 2; ++i) std::printf(" %ld %ld", reinterpret_cast<long>(a.w[i]), static_cast<long>(a.ld_w[i]));
    std::printf(" %ld\n", reinterpret_cast<long>(a.part));
    return hipSuccess;
}
}

// kind outputs rows cols hidden, then address and ld of d, d, h, w, w
int main(int argc, char** argv)
{
    if (argc != 16) return 2;
    const auto arg = [&](int i) { return std::strtoll(argv[i], nullptr, 10); };
    const auto at = [&](int i) { return reinterpret_cast<const uint16_t*>(arg(i)); };
    const FfnKind kind = static_cast<FfnKind>(arg(1));
    FfnArgs a{};
    a.rows = arg(3), a.cols = arg(4), a.hidden = arg(5);
    for (int i = 0; i < 2; ++i) a.d[i] = at(6 + 2 * i), a.ld_d[i] = arg(7 + 2 * i), a.w[i] = at(12 + 2 * i), a.ld_w[i] = arg(13 + 2 * i);
    a.h = at(10), a.ld_h = arg(11);
    for (int i = 0; i < arg(2); ++i) a.out[i].p = reinterpret_cast<void*>(uint64_t{1} << (52 + i));
    a.part = reinterpret_cast<float*>(kSpace);
    std::printf("space %ld %zu\n", static_cast<long>(kSpace), ffn_workspace_bytes(kind, a.rows, a.cols, a.hidden));
    return launch_ffn(kind, a, nullptr) == hipSuccess ? 0 : 1;
}
