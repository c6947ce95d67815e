// The host side of the library over stub launches: "device" memory is host
// memory, a plan's upload is a memcpy, and the fused step checks its plan as
// the kernels do. Built and run by test_block_workspace.py on the CPU.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "zero_block.h"
#include "zero_internal.h"
#include "zero_step.h"

namespace {
int uploads = 0;
bool plan_ok = false, table_ok = false;
zero::NormGradArgs grad{};
std::vector<uint8_t> table;  // as uploaded: the plan's workspace from byte 256, behind its header
uint8_t* table_at = nullptr;
bool table_whole() { return std::memcmp(table_at, table.data(), table.size()) == 0; }
}  // namespace

extern "C" {
hipError_t hipGetDevice(int* d)
{
    *d = 0;
    return hipSuccess;
}
}

namespace zero {

hipError_t launch_plan_write(uint8_t* ws, const WriteChunk& c, hipStream_t)
{
    ++uploads;
    std::memcpy(ws + c.offset, c.data, 4 * c.words);
    if (c.offset != 0) {
        table_at = ws + kAlign;
        table.resize(c.offset + 4 * c.words - kAlign);
        std::memcpy(table.data() + c.offset - kAlign, c.data, 4 * c.words);
    }
    return hipSuccess;
}
hipError_t launch_plan_tiles(const TensorDesc*, int, TileRef*, TileRef*, hipStream_t) { return hipSuccess; }
hipError_t launch_fused(Mode, int, const PlanHeader* hdr, const TensorDesc*, const TileRef*, int64_t, uint64_t sig, int, float,
                        const AdamScalars&, Partial*, const FinalizeArgs&, const zero_result*, hipStream_t)
{
    plan_ok = hdr->signature == sig;
    table_ok = table_whole();
    return hipSuccess;
}
int compute_units() { return 256; }

hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t)
{
    grad = a;
    // what the kernels write of the workspace
    const size_t sums = static_cast<size_t>(a.plan.units) * a.cols;
    const bool post = a.dw_post.p != nullptr || (a.plan.per_gate > 0 && a.dgate.p != nullptr);
    for (size_t i = 0; i < sums; ++i) {
        if (a.dw_pre.p != nullptr) a.sum_pre[i] = 1.5f;
        if (post) a.sum_post[i] = 2.5f;
    }
    for (int64_t i = 0; a.plan.strips > 0 && i < 2 * a.rows; ++i) a.row_sums[i] = 3.5f;
    return hipSuccess;
}
hipError_t launch_wgrad(const WgradArgs& a, const WgradPlan& plan, int, hipStream_t)
{
    std::memset(a.part, 0x3F, plan.bytes);
    return hipSuccess;
}
hipError_t launch_check(const float*, const Layout&, Partial* parts, int, hipStream_t)
{
    std::memset(static_cast<void*>(parts), 0x3F, 64);
    return hipSuccess;
}
hipError_t launch_finalize(const Partial*, int64_t, double, double, int, zero_result*, hipStream_t) { return hipSuccess; }
int resident_grid_check() { return 1; }

// the plans of the calls, small: the largest workspace here is a few MiB
WgradPlan wgrad_plan(int64_t, int64_t, int64_t) { return WgradPlan{2, 0, 4, 64, 4 * 64 * 64 * 4}; }
NormGradPlan norm_grad_plan(int64_t rows, int64_t cols, int64_t gate_rows)
{
    NormGradPlan p{};
    p.gates = gate_rows > 0 ? (rows + gate_rows - 1) / gate_rows : 1;
    p.gate_rows = gate_rows > 0 ? gate_rows : rows;
    if (gate_rows == 1) p.unit_gates = 1;
    else {
        p.per_gate = 1;
        p.unit_rows = p.gate_rows;
    }
    p.units = p.gates;
    p.strips = cols > 6144 ? 2 : 0;
    p.bytes = 2 * sizeof(float) * static_cast<size_t>(p.units * cols + (p.strips > 0 ? rows : 0));
    return p;
}

}  // namespace zero

namespace {

constexpr size_t kBytes = 8 << 20;
constexpr int kTensors = 700;  // 76 KiB of table: 8 rows of 8192 columns need 64 and their row sums
alignas(256) uint8_t memory[2 * kBytes];
alignas(16) uint8_t buffer[64];
const zero_rows kBf16{buffer, 1 << 14, ZERO_BF16, 0}, kF32{buffer, 1 << 14, ZERO_F32, 0};
zero_rows at(int i) { return zero_rows{buffer + 4 * i, 1 << 14, ZERO_F32, 0}; }

void step()
{
    const void* grads[1] = {buffer};
    zero_tensor t{};
    t.n = 8;
    t.grads = grads;
    t.master = t.exp_avg = t.exp_avg_sq = reinterpret_cast<float*>(buffer);
    t.param_out = buffer;
    const std::vector<zero_tensor> list(kTensors, t);
    zero_adamw_hparams hp{};
    hp.lr = 1e-3;
    hp.eps = 1e-8;
    hp.step = 1;
    hp.grad_scale = 1.0;
    zero_result r{};
    uploads = 0;
    if (zero_step(list.data(), kTensors, 1, &hp, 0.0, memory, kBytes, &r, nullptr) != ZERO_OK) std::abort();
}

// which: p, o, g: dw_pre, dw_post, dgate are asked for
int norm_grad(const char* which, int64_t cols, int64_t gate_rows, void* ws)
{
    zero_block_norm_grad_args g{};
    g.rows = 8;
    g.cols = cols;
    g.gate_rows = gate_rows;
    g.residual_scale = 1.0;
    g.dh = g.y = kBf16;
    g.w_pre = g.w_post = g.x_out = kF32;
    if (gate_rows > 0) g.gate = kF32;
    g.dx = at(8);
    g.rstd_pre = g.rstd_post = reinterpret_cast<float*>(buffer);
    if (std::strchr(which, 'p')) g.dw_pre = at(9);
    if (std::strchr(which, 'o')) g.dw_post = at(10);
    if (std::strchr(which, 'g')) g.dgate = at(11);
    return zero_block_norm_grad(&g, ws, kBytes, nullptr);
}

int run(const char* what, const char* which, int64_t cols, int64_t gate_rows, size_t offset)
{
    void* ws = memory + offset;
    if (std::strcmp(what, "norm_grad") == 0) return norm_grad(which, cols, gate_rows, ws);
    if (std::strcmp(what, "check") == 0) {
        zero_result r{};
        return zero_grad_check_norm(reinterpret_cast<float*>(buffer), 8, nullptr, 0.0, ws, kBytes, &r, nullptr);
    }
    return zero_act8_wgrad(&kBf16, buffer, 8, 8, 8, ZERO_ACT8_E4M3, nullptr, &kF32, 0, ws, kBytes, nullptr);
}

}  // namespace

// what which cols gate_rows offset: a step, one more, the call with its
// workspace `offset` bytes into the step's, and the step again. Prints the
// uploads of the three steps and whether the last found its plan and an intact
// table; then whether the call left the plan's signature and its table as they
// were, which is what a step whose launches were captured before it would meet.
int main(int argc, char** argv)
{
    if (argc != 6) return 2;
    const int64_t cols = std::atoll(argv[3]), gate_rows = std::atoll(argv[4]);
    const size_t offset = static_cast<size_t>(std::atoll(argv[5]));
    step();
    const int first = uploads;
    step();
    const int again = uploads;
    const auto* hdr = reinterpret_cast<const zero::PlanHeader*>(memory);
    const uint64_t signature = hdr->signature;
    if (run(argv[1], argv[2], cols, gate_rows, offset) != ZERO_OK) return 3;
    const bool signature_kept = hdr->signature == signature;
    const bool table_kept = table_whole();
    step();
    std::printf("%d %d %d %d %d %d %d\n", first, again, uploads, plan_ok, table_ok, signature_kept, table_kept);
    return 0;
}
