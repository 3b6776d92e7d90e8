// tree_launch.h -- into how many slices a launch of the tree attention cuts its lists (host code
// without CUDA).
#pragma once

#include <atomic>

namespace ssa {

constexpr int kMaxSlices = 8;

// What the devices answered for one kernel: clusters of k CTAs that run at once, plus 1; 0 is not
// asked yet.
struct ClusterCounts {
    static constexpr int kDevices = 64;
    std::atomic<int> n[kDevices][kMaxSlices + 1];
};

// The largest number of slices (CTAs of a cluster), at most `most`, with which `items` clusters run
// at once on the device.  query(k): clusters of k CTAs that it runs, or less than 0 if it does not say,
// which is taken as none for this call and asked again by the next.
template <class Query>
int pick_slices(ClusterCounts &counts, int device, long long items, int most, Query query) {
    for (int k = most < kMaxSlices ? most : kMaxSlices; k > 1; --k) {
        const bool keep = device >= 0 && device < ClusterCounts::kDevices;
        int n = keep ? counts.n[device][k].load() : 0;
        if (n == 0) {
            n = query(k) + 1;
            if (n < 1) continue;
            if (keep) counts.n[device][k].store(n);
        }
        if (items <= n - 1) return k;
    }
    return 1;
}

}  // namespace ssa
