// The list of places by the kernels' own rule (sight.cuh), on the host: lines of T L window sinks box_log in; out for each
// s1 i1 end lo tail, then, where `end` is under a million, every place's position and whether some token sees it, then the
// positions of the two places past the end.
#include <cstdio>

#include "sight.cuh"

int main() {
    int T, L, window, sinks, box_log;
    while (std::scanf("%d %d %d %d %d", &T, &L, &window, &sinks, &box_log) == 5) {
        const specv::Sight s(T, L, window, sinks, box_log);
        std::printf("%d %d %d %d %d", s.s1, s.i1, s.end, s.lo, s.tail);
        if (s.end < 1000000)
            for (int i = 0; i < s.end; ++i) std::printf(" %d %d", s.at(i), (int)s.seen(s.at(i), L, sinks));
        std::printf(" %d %d\n", s.at(s.end), s.at(s.end + 1));
    }
}
