// The host side of the language-model operators with the HIP runtime replaced by a recorder: entry points, plans and
// launch code are the library's own, compiled for the host alone; a launch is written down and nothing runs.
// Compiled and driven by lm_launches.py.
#include "../allgather_gemm_amd/csrc/ag_internal.hpp"
#include "../allgather_gemm_amd/csrc/lm_tile.hpp"

#include <iterator>
#include <map>
#include <string>
#include <vector>

namespace {

struct Launch {
    std::string name;
    int64_t grid[3], block[3];
    bool tile;                 // its argument is a TileArgs
    ag::lm::TileArgs args;
};

std::map<const void*, std::string>& names()
{
    static std::map<const void*, std::string> m;
    return m;
}
std::vector<Launch> g_launches;
dim3 g_grid, g_block;
int g_cus = 256;

}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*)
{
    static void* handle;
    return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char* device, const char*, unsigned, void*, void*, void*, void*, int*)
{
    names()[host] = device;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t)
{
    g_grid = grid;
    g_block = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream)
{
    *grid = g_grid;
    *block = g_block;
    *shared = 0;
    *stream = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t)
{
    Launch l = {names()[f], {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}, false, {}};
    l.tile = l.name.find("TileArgs") != std::string::npos;
    if (l.tile)
        l.args = *static_cast<const ag::lm::TileArgs*>(args[0]);
    g_launches.push_back(l);
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }

void rec_start(int cus)
{
    g_cus = cus;
    g_launches.clear();
}
int rec_count() { return (int)g_launches.size(); }
const char* rec_name(int i) { return g_launches[i].name.c_str(); }
void rec_dims(int i, int64_t* out)
{
    for (int k = 0; k < 3; ++k) {
        out[k] = g_launches[i].grid[k];
        out[3 + k] = g_launches[i].block[k];
    }
}
// M, N, K, group, E, splits, whether it writes fp32 sums, whether it adds to them; false where it has no TileArgs
int rec_args(int i, int64_t* out)
{
    const ag::lm::TileArgs& a = g_launches[i].args;
    const int64_t v[8] = {a.M, a.N, a.K, a.group, a.E, a.splits, a.part != nullptr, a.accumulate};
    for (int k = 0; k < 8; ++k)
        out[k] = v[k];
    return g_launches[i].tile;
}

// Every kernel that the library has, as the runtime is told of it.
int rec_kernels() { return (int)names().size(); }
const char* rec_kernel(int i) { return std::next(names().begin(), i)->second.c_str(); }

// How a 256 x 256 kernel cuts what n units of a tile's time and `lone` halves leave for a last round
void rec_tail(int n, int lone, int columns, int quarter_columns, int workgroups, int* out)
{
    const ag::lm::Tail t = ag::lm::tail_of(n, lone, columns, quarter_columns, workgroups);
    out[0] = t.cut;
    out[1] = t.quarters;
}
int rec_big_rows(int n) { return ag::lm::big_rows<256, true>(n); }
int rec_half_rows(int n) { return ag::lm::half_rows<256, true>(n); }

}  // extern "C"

namespace ag {

hipError_t device_cus(int* out)
{
    *out = g_cus;
    return hipSuccess;
}
int hip_error(hipError_t, const char*) noexcept { return -3; }

}  // namespace ag
