"""What the gated linear recurrence keeps about a device, with host threads that come to it at the same time: a program of threads around
the header, whose look-ups wait for one another where the order counts."""
import subprocess

from linear_attention_chunkwise_gb300 import _build

PROGRAM = r"""
#include <atomic>
#include <cstdio>
#include <initializer_list>
#include <thread>
#include "kda_glr_room.h"

using namespace kda;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

GlrRooms rooms, crowded;

bool is(const GlrRoom& r, int value) {
    for (int n = 0; n <= kGlrMaxCluster; ++n)
        if (r.clusters[n] != value) return false;
    return true;
}
struct Look {
    int value, error;
    std::atomic<int>* count;
    int operator()(GlrRoom* r) const {
        if (count) ++*count;
        for (int& c : r->clusters) c = value;
        return error;
    }
};

int main() {
    // A thread that began to look before the device was known ends after others have what was kept.
    std::atomic<int> began{0}, go{0}, late{0};
    GlrRoom slow_room;
    std::thread slow([&] {
        const auto look = [&](GlrRoom* r) {
            for (int n = 0; n <= kGlrMaxCluster; ++n) {
                r->clusters[n] = 9;
                if (n == 3) {
                    began = 1;
                    while (!go) std::this_thread::yield();
                }
            }
            return 0;
        };
        late = rooms.get(5, look, &slow_room);
    });
    while (!began) std::this_thread::yield();
    GlrRoom first, then;
    std::atomic<int> count{0};
    CHECK(rooms.get(5, Look{7, 0, &count}, &first) == 0 && is(first, 7));
    CHECK(rooms.get(5, Look{8, 0, &count}, &then) == 0 && is(then, 7) && count == 1);
    go = 1;
    slow.join();
    CHECK(late == 0 && is(slow_room, 9));  // its own look-up is its own call's
    CHECK(rooms.get(5, Look{8, 0, &count}, &then) == 0 && is(then, 7) && count == 1);

    // An error is the caller's and is not kept.
    CHECK(rooms.get(6, Look{1, 3, nullptr}, &then) == 3);
    CHECK(rooms.get(6, Look{2, 0, nullptr}, &then) == 0 && is(then, 2));

    // Devices without a place look each time, and are nobody else's.
    for (const int dev : {64, 69, 1000}) {
        count = 0;
        CHECK(rooms.get(dev, Look{4, 0, &count}, &then) == 0 && is(then, 4));
        CHECK(rooms.get(dev, Look{3, 0, &count}, &then) == 0 && is(then, 3) && count == 2);
    }
    CHECK(rooms.get(5, Look{8, 0, nullptr}, &then) == 0 && is(then, 7));

    // Many at once: every call has one look-up's table, whole, and later calls the same one.
    std::thread threads[16];
    std::atomic<int> torn{0};
    for (int t = 0; t < 16; ++t)
        threads[t] = std::thread([&, t] {
            for (int i = 0; i < 20000; ++i) {
                GlrRoom r;
                const int dev = i % 64;
                crowded.get(dev, Look{t, 0, nullptr}, &r);
                if (!is(r, r.clusters[0])) ++torn;
            }
        });
    for (auto& t : threads) t.join();
    CHECK(torn == 0);
    return 0;
}
"""


def test_host_threads_that_come_together(tmp_path):
    (tmp_path / "rooms.cpp").write_text(PROGRAM)
    program = str(tmp_path / "rooms")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-pthread", "-I", _build.CSRC, "-o", program,
                    str(tmp_path / "rooms.cpp")], check=True)
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
