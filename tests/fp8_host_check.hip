// Host-only check of what the block-scaled FP8 calls and the group norm hand to
// their kernels (built and run by tests/test_fp8_host.py; no GPU code is
// executed): the library's own host code with the HIP runtime's queries and
// launches replaced by recorders.  One line is printed for each disagreement, and
// the exit status says whether there was any.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

namespace fake {
int device = 0;
struct Launch {
  const void* kernel;
  dim3 grid, block;
  size_t lds;
};
std::vector<Launch> launches;
template <typename A>
struct Args {
  static A last;  // of the kernels that take an A first
};
template <typename A>
A Args<A>::last{};

hipError_t get_device(int* d) {
  *d = device;
  return hipSuccess;
}
hipError_t get_properties(hipDeviceProp_t* p, int) {
  memset(p, 0, sizeof(*p));
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t last_error() { return hipSuccess; }
// a kernel's limit of dynamic and static LDS, on each device
std::map<std::pair<int, const void*>, int> lds_limits;
std::mutex lds_mutex;
hipError_t set_attribute(const void* kernel, hipFuncAttribute what, int value) {
  if (what != hipFuncAttributeMaxDynamicSharedMemorySize) return hipErrorInvalidValue;
  std::lock_guard<std::mutex> lk(lds_mutex);
  lds_limits[{device, kernel}] = value;
  return hipSuccess;
}
int lds_limit(const void* kernel) {
  const auto it = lds_limits.find({device, kernel});
  return it == lds_limits.end() ? 64 << 10 : it->second;
}
template <typename A, typename... More>
void launch(const void* kernel, dim3 grid, dim3 block, size_t lds, const A& a, const More&...) {
  launches.push_back(Launch{kernel, grid, block, lds});
  Args<A>::last = a;
}
}  // namespace fake

#undef hipGetDeviceProperties
#define hipGetDeviceProperties fake::get_properties
#define hipFuncSetAttribute fake::set_attribute
#define hipGetDevice fake::get_device
#define hipGetLastError fake::last_error
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  fake::launch(reinterpret_cast<const void*>(kernel), grid, block, lds, __VA_ARGS__)

#include "rq_api.hip"
#include "rq_gemm_fp8.hip"
#include "rq_groupnorm.hip"
#include "rq_quant.hip"

namespace {
int bad = 0;
void expect(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0) {
  if (!ok) printf("WRONG %s: %lld %lld %lld\n", what, a, b, c), bad++;
}
template <typename T>
T* array_at(size_t i) {
  return reinterpret_cast<T*>((size_t)0x100000000000 + (i << 38));
}
// one launch, within a launch's limits and its kernel's LDS
const fake::Launch& launched(const char* what, long long a, long long b, long long c) {
  static const fake::Launch none{};
  expect(fake::launches.size() == 1, what, a, b, c);
  if (fake::launches.empty()) return none;
  const fake::Launch& l = fake::launches.back();
  for (int axis = 0; axis < 2; axis++) {
    const size_t n = axis ? (size_t)l.grid.y * l.block.y : (size_t)l.grid.x * l.block.x;
    expect(n > 0 && n < (size_t)1 << 32, "work-items of an axis", a, b, c);
  }
  expect((int)l.lds <= fake::lds_limit(l.kernel), "LDS within its limit", a, b, c);
  return l;
}
}  // namespace

// Every kernel has sizes that take it.
int taken[rq::FP64 + 1][3];

static void products() {
  const int ms[] = {1, 2, 4, 5, 8, 16, 17, 32, 33, 61, 64, 65, 100, 128, 129, 200, 256, 300, 511, 512,
                    700, 1000, 1100, 1500, 2047, 2048, 2500, 4001, 4352, 10000, 1 << 20, 1 << 24};
  const int ns[] = {1, 7, 128, 256, 768, 1000, 1024, 1152, 2048, 2560, 4096, 8192, 16384, 65529, 65536,
                    1 << 20, 1 << 24};
  const int ks[] = {128, 256, 768, 1024, 2560, 4096, 16384, 1 << 22};
  for (int m : ms)
    for (int n : ns)
      for (int k : ks) {
        // outputs within their limit, operands within their part of the addresses
        if ((long long)m * n > RQ_FP8_MAX_VALUES || (long long)m * k >> 38 || (long long)n * k >> 38) continue;
        for (int count : {1, 3, 8}) {
          rq_fp8_problem p[8];
          rq::Fp8Args a{};
          a.count = count;
          a.M = m;
          for (int i = 0; i < count; i++) {
            p[i] = {array_at<void>(0), array_at<void>(1), array_at<void>(2), array_at<void>(3), nullptr,
                    array_at<void>(10 + 2 * i), array_at<void>(11 + 2 * i), n, k};
            a.p[i].N = n;
            a.p[i].K = k;
          }
          rq::Plan plans[2][2];
          for (int out = 0; out < 3; out++) {
            if (out == RQ_TYPE_E4M3 && n % 128) continue;
            for (int scale = 0; scale < 2; scale++) {
              size_t bytes = 0;
              expect(rq_gemm_fp8_workspace_size(p, count, m, scale, out, &bytes) == RQ_OK, "size", m, n, k);
              expect(bytes <= (size_t)RQ_GEMM_WORKSPACE_MAX_BYTES, "most bytes", m, n, k);
              for (int ws = 0; ws < 2; ws++) {
                a.out = out;
                const rq::Plan c = rq::choose(a, ws != 0);
                taken[c.kind][out]++;
                if (out) plans[out - 1][ws] = c;
                expect(c.splits > 1 ? ws && bytes == rq::plan_bytes(a, c) : !ws || !bytes, "workspace", m, n, k);
                expect(c.splits <= k / 128, "ranges of K", m, n, k);
                for (fake::device = 0; fake::device < 2; fake::device++) {
                  fake::launches.clear();
                  expect(rq_gemm_fp8(p, count, m, scale, out, RQ_ACT_NONE, ws ? array_at<void>(9) : nullptr,
                                     ws ? (size_t)RQ_GEMM_WORKSPACE_MAX_BYTES : 0, nullptr) == RQ_OK,
                         "call", m, n, k);
                  const fake::Launch& l = launched("launches of a product", m, n, k);
                  expect((long long)l.grid.x == rq::tiles_of(a, c.kind) * c.splits, "grid", m, n, k);
                  const rq::Shape& t = rq::SHAPES[c.kind];
                  expect(rq::tiles_of(a, c.kind) ==
                             (long long)count * ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn),
                         "tiles", m, n, k);
                  expect(c.kind > rq::ROWS64 || m <= 16, "rows", m, n, k);
                }
                fake::device = 0;
              }
            }
          }
          // binary16 and E4M3 outputs add in one order: rows and rings all do
          if (n % 128 == 0)
            for (int ws = 0; ws < 2; ws++) {
              const rq::Plan &h = plans[0][ws], &q = plans[1][ws];
              expect((h.kind <= rq::RING8X2 && q.kind <= rq::RING8X2) ||
                         (h.kind == q.kind && h.splits == q.splits && h.kind >= rq::FP128),
                     "order of sums", m, n, k);
            }
        }
      }
}

static void rows() {
  for (int m : {1, 3, 1000, 1 << 20, 1 << 24})
    for (int k : {128, 1024, 16384, 1 << 22}) {
      if ((long long)m * k > RQ_FP8_MAX_VALUES) continue;
      for (int half = 0; half < 2; half++) {
        fake::launches.clear();
        expect(rq_quant_fp8(array_at<void>(0), half, RQ_ACT_RELU2, array_at<void>(1), array_at<void>(2),
                            RQ_SCALE_F32, m, k, nullptr) == RQ_OK,
               "quant", m, k);
        const fake::Launch& l = launched("launches of quant", m, k, 0);
        expect((size_t)l.grid.x * l.block.x * 8 >= (size_t)m * k, "every value", m, k);
      }
    }
}

static void norms() {
  for (int t : {1, 3, 1000, (1 << 23) + 5, 1 << 24})
    for (int c : {32, 256, 1024, 4096, 1 << 20})
      for (int size : {32, 256}) {
        if ((long long)t * c > RQ_FP8_MAX_VALUES || c % size) continue;
        rq_groupnorm_args g{};
        g.y = array_at<const float>(0);
        g.out = array_at<void>(1);
        g.T = t;
        g.C = c;
        g.groups = c / size;
        fake::launches.clear();
        expect(rq_groupnorm(&g, nullptr) == RQ_OK, "norm", t, c, size);
        const fake::Launch& l = launched("launches of a norm", t, c, size);
        const size_t lanes = (size_t)l.grid.x * l.grid.y * l.block.x;
        expect(lanes * 4 >= (size_t)t * c && (l.grid.y == 1 || l.grid.y == 2), "every channel", t, c, size);
      }
}

int main() {
  products();
  for (int k = 0; k <= rq::FP64; k++) {
    const bool quantized = k == rq::RING8X1 || k == rq::RING8X2 || k >= rq::FP128;
    const bool binary32 = k < rq::RING8X1 || k == rq::WIDE64 || k == rq::WIDE128;
    const bool binary16 = k < rq::RING8X1 || k >= rq::FP128;
    expect(!binary32 == !taken[k][0] && !binary16 == !taken[k][1] && !quantized == !taken[k][2],
           "sizes of a kernel", k);
  }
  rows();
  norms();
  printf("wrong=%d\n", bad);
  return bad != 0;
}
